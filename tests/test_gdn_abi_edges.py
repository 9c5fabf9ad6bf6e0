"""Host-side checks of the gated delta rule's calls, without a GPU: what only some of them take."""
import ctypes

import pytest

from chunked_kimi_delta_gb300 import KDA_ZERO_BEHIND, kda_fwd_args
from test_gdn_lora_abi import BASE, FWD, INVALID, WORKSPACE, _bwd, _fill, _fwd, _step, lib  # noqa: F401


@pytest.mark.parametrize("kw", [dict(out=BASE), dict(out=2 * BASE)])
def test_step_refuses_a_result_over_queries_or_keys(lib, kw):  # noqa: F811
    """The CTAs of a head's value channels, and of a key head's group, read them at no fixed time."""
    assert lib.kda_gdn_recurrent_step(ctypes.byref(_step(**kw)), None) == INVALID


def test_the_chunked_calls_alone_zero_what_is_behind(lib):  # noqa: F811
    flags = FWD["flags"] | KDA_ZERO_BEHIND
    assert lib.kda_gdn_chunk_fwd(ctypes.byref(_fwd(flags=flags, workspace=None)), None) == WORKSPACE
    assert lib.kda_gdn_chunk_bwd(ctypes.byref(_bwd(dict(flags=flags), workspace=None)), None) == WORKSPACE
    assert lib.kda_gdn_recurrent_step(ctypes.byref(_step(flags=KDA_ZERO_BEHIND)), None) == INVALID
    a = _fill(kda_fwd_args(), FWD, flags=flags, Hk=4)
    assert lib.kda_chunk_fwd(ctypes.byref(a), None) == INVALID
