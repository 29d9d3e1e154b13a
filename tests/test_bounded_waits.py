"""Every wait for an mbarrier ends: the kernels' sources wait through functions that go by the
timer, and those give up after the limit, the second of two waiters on the flag that the
first one raised."""
import ctypes
import glob
import os
import re

import pytest
import torch

import attention_attn_varlen_gb300 as av

CSRC = os.path.join(os.path.dirname(av.__file__), "csrc")
ERR_TIMEOUT, SRC_SELFTEST = 1 << 1, 1 << 13


def _code(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


def test_barriers_are_polled_in_timed_waits_alone():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        name, code = os.path.basename(path), _code(path)
        polls = len(re.findall(r"\bmbar_try_wait\s*\(|mbarrier\.(?:try|test)_wait", code))
        # common.cuh: the try itself, mbar_wait and its slow path; chunks.cuh: chunk_wait, chunk_wait_each
        assert polls == {"common.cuh": 4, "chunks.cuh": 2}.get(name, 0), name
    for name, function in (("common.cuh", "mbar_wait_slow"), ("chunks.cuh", "chunk_wait"),
                           ("chunks.cuh", "chunk_wait_each")):
        code = _code(os.path.join(CSRC, name))
        body = code[code.index(f"bool {function}("):]
        body = body[:body.index("\n}")]
        assert "globaltimer" in body and re.search(r"kWaitLimitNs|>> 30", body) and re.search(r"\*abort\b", body), function


def test_the_self_tests_need_a_place_for_their_result():
    av.build()
    for delta in (0, 1):
        assert av.lib().attn_selftest_chunk_wait(None, delta, None) == 1
        if not torch.cuda.is_available():
            assert av.lib().attn_selftest_chunk_wait(None, delta, (ctypes.c_ulonglong * 4)()) == 7
    with pytest.raises(ValueError):
        av.selftest_bounded_wait(wait="none")


@pytest.mark.gpu
@pytest.mark.parametrize("wait", ["linear", "delta"])
def test_a_chunk_kernels_wait_gives_up_and_the_context_stays_usable(wait):
    av.get_last_device_error()
    r = av.selftest_bounded_wait(wait=wait)
    assert not r["first_ok"] and 0.9e9 <= r["first_ns"] <= 3.0e9, r          # a limit of one second
    assert not r["second_ok"] and r["second_ns"] < 0.9e9, r                  # started half a limit later
    st, word = av.get_last_device_error()
    assert st == 5 and word == ERR_TIMEOUT | SRC_SELFTEST, hex(word)
    # the chunk kernels run as before
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(200, 2, 64, generator=gen, device="cuda").bfloat16() for _ in range(3))
    g = -torch.rand(200, 2, generator=gen, device="cuda")
    cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    runs = [av.delta_attn_varlen_fwd(q, k, v, g, -g, cu, 200, qk_norm_eps=1e-6) for _ in range(2)]
    assert torch.equal(*runs) and torch.isfinite(runs[0].float()).all()
    assert av.get_last_device_error() == (0, 0)
