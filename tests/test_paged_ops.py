"""The operators around the paged cache without a GPU: arguments that are refused, calls with
nothing to do, the rotary frequencies, and the 64-bit forms that the GPU tests hold the kernels
to."""
import math
import os
import subprocess

import pytest
import torch

import paged_ref as ref
from fp8_attention_forward_gb300 import build, fa8
from paged_ref import E4M3, Problem, e4m3, val

BAD, UNSUPPORTED, CUDA = fa8.FA8_ERR_INVALID_ARG, fa8.FA8_ERR_UNSUPPORTED, fa8.FA8_ERR_CUDA


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    fa8.lib()


def e8(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(E4M3)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def f32(*shape):
    return torch.ones(shape, dtype=torch.float32)


def status(fn, args, change):
    """The status of the call with some arguments changed (no GPU here: a valid call gets as far as CUDA)."""
    a = dict(args, **change)
    pos = [a.pop(n) for n in fn.order]
    try:
        fn(*pos, **a)
    except fa8.Fa8Error as e:
        assert e.status == fa8.FA8_SUCCESS or str(e)
        return e.status
    return fa8.FA8_SUCCESS


fa8_rope, fa8_bounds, fa8_select, fa8_fwd = (lambda *a, _f=f, **k: _f(*a, **k) for f in (
    fa8.rope_append, fa8.page_bounds, fa8.select_pages, fa8.fwd_pages))
fa8_rope.order, fa8_bounds.order = ["q", "k", "v", "inv_freq"], ["k", "bounds"]
fa8_select.order, fa8_fwd.order = ["q", "bounds", "top_k"], ["q", "k", "v", "pages"]
TABLE = dict(cu_seqlens_k=i32(3), block_table=i32(2, 5), page_size=16)


def qkv16(lead=(2, 3), Hq=8, Hkv=2, D=128, DV=128, dt=torch.bfloat16):
    return dict(q=torch.zeros((*lead, Hq, D), dtype=dt), k=torch.zeros((*lead, Hkv, D), dtype=dt),
                v=torch.zeros((*lead, Hkv, DV), dtype=dt))


ROPE = dict(qkv16(), inv_freq=torch.ones(64, dtype=torch.float64), k_out=e8(9, 16, 2, 128), v_out=e8(9, 16, 2, 128), **TABLE)
PACKED = dict(qkv16((6,)), cu_seqlens_q=i32(3))


@pytest.mark.parametrize("change,want", [
    ({}, CUDA), (PACKED, CUDA),
    (dict(k_out=e8(2, 7, 2, 128), v_out=e8(2, 7, 2, 128), cu_seqlens_k=None, block_table=None), CUDA),
    (dict(k_out=e8(7, 2, 128), v_out=e8(7, 2, 128), block_table=None), CUDA),
    (dict(inv_freq=torch.ones(8)), CUDA), (dict(positions=i32(2, 3)), CUDA),
    (qkv16((2, 0)), fa8.FA8_SUCCESS), (dict(qkv16((0,)), cu_seqlens_q=i32(3)), fa8.FA8_SUCCESS),
    (qkv16(dt=torch.float32), UNSUPPORTED), (dict(k=torch.zeros((2, 3, 2, 128), dtype=torch.float16)), BAD),
    (dict(k=torch.zeros((2, 2, 2, 128), dtype=torch.bfloat16)), BAD),
    (dict(k=torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16)), BAD),
    (dict(k=torch.zeros((2, 3, 3, 128), dtype=torch.bfloat16), v=torch.zeros((2, 3, 3, 128), dtype=torch.bfloat16)), BAD),
    (qkv16(D=80, DV=80), UNSUPPORTED), (dict(q=torch.zeros((2, 3, 8, 256), dtype=torch.bfloat16)[..., ::2]), BAD),
    (dict(q=torch.zeros((2, 3, 8, 132), dtype=torch.bfloat16)[..., :128]), BAD),
    (dict(q=torch.zeros((2, 3, 8, 136), dtype=torch.bfloat16)[..., 1:129]), BAD),
    (qkv16((6,)), BAD), (dict(cu_seqlens_q=i32(3)), BAD), (dict(PACKED, cu_seqlens_q=i32(1)), BAD),
    (dict(inv_freq=torch.ones(72, dtype=torch.float64)), BAD), (dict(inv_freq=torch.ones(60, dtype=torch.float64)), UNSUPPORTED),
    (dict(inv_freq=torch.ones(64, dtype=torch.bfloat16)), BAD), (dict(inv_freq=torch.ones(0)), BAD),
    (dict(inv_freq=torch.ones(32), rotary_offset=72), BAD), (dict(inv_freq=torch.ones(32), rotary_offset=4), UNSUPPORTED),
    (dict(rotary_offset=-8), UNSUPPORTED), (dict(rot_scale=math.inf), BAD),
    (dict(positions=i32(2, 4)), BAD), (dict(positions=f32(2, 3)), BAD), (dict(positions=i32(6)), BAD),
    (dict(descale_q=f32(2, 3)), BAD), (dict(descale_k=i32(2, 2)), BAD),
    (dict(k_out=torch.zeros((9, 16, 2, 128), dtype=torch.bfloat16)), UNSUPPORTED),
    (dict(k_out=e8(9, 16, 3, 128)), BAD), (dict(v_out=e8(8, 16, 2, 128)), BAD), (dict(v_out=e8(9, 16, 2, 64)), BAD),
    (dict(k_out=e8(9, 16, 2, 136)[..., :128]), BAD), (dict(q_out=e8(2, 3, 8, 64)), BAD), (dict(q_out=e8(6, 8, 128)), BAD),
    (dict(page_size=8), BAD), (dict(block_table=i32(3, 5)), BAD), (dict(block_table=f32(2, 5)), BAD),
    (dict(block_table=i32(5, 2).T), BAD), (dict(cu_seqlens_k=None), BAD), (dict(cu_seqlens_k=i32(4)), BAD),
    (dict(block_table=None), BAD), (dict(k_out=e8(9, 12, 2, 128), v_out=e8(9, 12, 2, 128), page_size=12), UNSUPPORTED),
])
def test_rope_append_arguments(change, want):
    assert status(fa8_rope, ROPE, change) == want


BOUNDS = dict(k=e8(9, 16, 2, 128), bounds=e8(9, 2, 2, 128), **TABLE)


@pytest.mark.parametrize("change,want", [
    ({}, CUDA), (dict(new_tokens=4), CUDA), (dict(cu_seqlens_q=i32(3)), CUDA), (dict(new_tokens=0), fa8.FA8_SUCCESS),
    (dict(k=torch.zeros((9, 16, 2, 128), dtype=torch.bfloat16)), UNSUPPORTED),
    (dict(bounds=torch.zeros((9, 2, 2, 128), dtype=torch.bfloat16)), UNSUPPORTED),
    (dict(k=e8(9, 2, 128)), BAD), (dict(k=e8(9, 16, 2, 24), bounds=e8(9, 2, 2, 24)), BAD),
    (dict(k=e8(9, 16, 2, 272), bounds=e8(9, 2, 2, 272)), UNSUPPORTED),
    (dict(bounds=e8(8, 2, 2, 128)), BAD), (dict(bounds=e8(9, 3, 2, 128)), BAD), (dict(bounds=e8(9, 2, 3, 128)), BAD),
    (dict(bounds=e8(9, 2, 2, 144)[..., :128]), BAD), (dict(cu_seqlens_q=i32(4)), BAD),
    (dict(page_size=32), BAD), (dict(block_table=None), BAD), (dict(cu_seqlens_k=None), BAD),
])
def test_page_bounds_arguments(change, want):
    assert status(fa8_bounds, BOUNDS, change) == want


SELECT = dict(q=e8(2, 3, 8, 128), bounds=e8(9, 2, 2, 128), top_k=4, **TABLE)


@pytest.mark.parametrize("change,want", [
    ({}, CUDA), (dict(q=e8(6, 8, 128), cu_seqlens_q=i32(3)), CUDA), (dict(q=e8(2, 0, 8, 128)), fa8.FA8_SUCCESS),
    (dict(top_k=4096, keep_first=4000, keep_last=96), CUDA), (dict(block_table=i32(2, 16384)), CUDA),
    (dict(q=torch.zeros((2, 3, 8, 128), dtype=torch.bfloat16)), UNSUPPORTED),
    (dict(q=e8(2, 3, 8, 32), bounds=e8(9, 2, 2, 32)), UNSUPPORTED), (dict(q=e8(2, 3, 8, 64)), BAD), (dict(q=e8(2, 3, 7, 128)), BAD),
    (dict(q=e8(2, 3, 8, 136)[..., :128]), BAD), (dict(q=e8(6, 8, 128)), BAD), (dict(q=e8(2, 3, 258, 128)), UNSUPPORTED),
    (dict(top_k=0, keep_first=0, keep_last=0), BAD), (dict(top_k=4097), UNSUPPORTED), (dict(keep_first=-1), BAD),
    (dict(keep_first=3, keep_last=2), BAD), (dict(keep_last=2 ** 31 - 1, keep_first=2 ** 31 - 1), BAD),
    (dict(pages=i32(2, 3, 3, 4)), BAD), (dict(pages=f32(2, 3, 2, 4)), BAD), (dict(pages=i32(6, 2, 4)), BAD),
    (dict(pages=i32(2, 3, 4, 2).transpose(2, 3)), BAD), (dict(block_table=i32(2, 16385)), UNSUPPORTED),
    (dict(block_table=i32(3, 5)), BAD), (dict(cu_seqlens_k=i32(2)), BAD), (dict(page_size=4), UNSUPPORTED),
])
def test_select_pages_arguments(change, want):
    assert status(fa8_select, SELECT, change) == want


FWD = dict(q=e8(2, 3, 8, 128), k=e8(9, 16, 2, 128), v=e8(9, 16, 2, 128), pages=i32(2, 3, 2, 4), **TABLE)


@pytest.mark.parametrize("change,want", [
    ({}, CUDA), (dict(q=e8(6, 8, 128), pages=i32(6, 2, 4), cu_seqlens_q=i32(3)), CUDA), (dict(pages=i32(2, 3, 2, 0)), CUDA),
    (dict(q=e8(2, 0, 8, 128), pages=i32(2, 0, 2, 4)), fa8.FA8_SUCCESS), (dict(pages=i32(2, 3, 2, 4096)), CUDA),
    (dict(q=torch.zeros((2, 3, 8, 128), dtype=torch.float8_e5m2)), UNSUPPORTED), (dict(k=e8(9, 16, 2, 64)), BAD),
    (dict(v=e8(9, 16, 2, 64)), UNSUPPORTED), (dict(v=e8(8, 16, 2, 128)), BAD), (dict(k=e8(9, 2, 128)), BAD),
    (dict(v=e8(9, 2, 128)), BAD), (dict(q=e8(2, 3, 7, 128)), BAD), (dict(q=e8(2, 3, 258, 128)), UNSUPPORTED),
    (dict(pages=i32(2, 3, 2, 4097)), UNSUPPORTED), (dict(pages=i32(2, 3, 1, 4)), BAD), (dict(pages=i32(2, 2, 2, 4)), BAD),
    (dict(pages=f32(2, 3, 2, 4)), BAD), (dict(pages=i32(2, 3, 4, 2).transpose(2, 3)), BAD),
    (dict(out_dtype=torch.float32), BAD), (dict(out=torch.zeros((2, 3, 8, 64), dtype=torch.bfloat16)), BAD),
    (dict(out=torch.zeros((2, 3, 8, 132), dtype=torch.bfloat16)[..., :128]), BAD), (dict(lse=f32(2, 3, 8)), BAD),
    (dict(lse=torch.zeros((2, 8, 3), dtype=torch.float64)), BAD), (dict(sink=f32(7)), BAD), (dict(softmax_scale=math.nan), BAD),
    (dict(descale_q=f32(3, 2)), BAD), (dict(page_size=32), BAD), (dict(block_table=i32(1, 5)), BAD),
    (dict(k=e8(2, 4104, 2, 128), v=e8(2, 4104, 2, 128), page_size=4104), UNSUPPORTED), (dict(cu_seqlens_k=i32(9)), BAD),
])
def test_fwd_pages_arguments(change, want):
    assert status(fa8_fwd, FWD, change) == want


# ------------------------------------------------------------------ rotary frequencies
def test_rope_inv_freq_forms():
    R, base, L, f = 64, 10000.0, 4096, 8.0
    i = torch.arange(R // 2, dtype=torch.float64)
    w = base ** (-2 * i / R)
    close = dict(rtol=1e-14, atol=0)
    torch.testing.assert_close(fa8.rope_inv_freq(R, base), w, **close)
    torch.testing.assert_close(fa8.rope_inv_freq(R, base, scaling="linear", factor=f), w / f, **close)
    torch.testing.assert_close(fa8.rope_inv_freq(R, base, scaling="ntk", factor=f),
                               (base * f ** (R / (R - 2))) ** (-2 * i / R), **close)
    # NTK leaves the highest frequency and divides the lowest by factor
    ntk = fa8.rope_inv_freq(R, base, scaling="ntk", factor=f)
    assert ntk[0] == 1 and abs(ntk[-1] * f / w[-1] - 1) < 1e-12
    turns = L * w / (2 * math.pi)
    bands = fa8.rope_inv_freq(R, base, scaling="bands", factor=f, original_len=L)
    keep = ((turns - 1) / (4 - 1)).clamp(0, 1)
    torch.testing.assert_close(bands, w * keep + w / f * (1 - keep), **close)
    assert (keep == 1).any() and (keep == 0).any() and ((keep > 0) & (keep < 1)).any()
    yarn = fa8.rope_inv_freq(R, base, scaling="yarn", factor=f, original_len=L)
    lo, hi = (R * math.log(L / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32, 1))
    keep = 1 - ((i - math.floor(lo)) / (math.ceil(hi) - math.floor(lo))).clamp(0, 1)
    torch.testing.assert_close(yarn, w * keep + w / f * (1 - keep), **close)
    assert yarn[0] == w[0] and yarn[-1] == w[-1] / f


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=7), dict(base=1.0), dict(base=math.inf),
                                dict(scaling="linear", factor=0.5), dict(scaling="yarn", factor=2.0),
                                dict(scaling="bands", factor=2.0, original_len=4096, low=4.0, high=4.0),
                                dict(scaling="linear", factor=math.nan), dict(scaling="ntk", factor=2.0, rotary_dim=2)])
def test_rope_inv_freq_refusals(kw):
    with pytest.raises(fa8.Fa8Error) as e:
        fa8.rope_inv_freq(**dict(dict(rotary_dim=64), **kw))
    assert e.value.status == BAD
    with pytest.raises(ValueError):
        fa8.rope_inv_freq(64, scaling="other")


# ------------------------------------------------------------------ the 64-bit forms themselves
def test_bound_is_an_upper_bound_of_every_key():
    p = Problem([100, 33], [1, 1], Hq=4, Hkv=2, D=64, DV=64, ps=8, seed=30)
    b, q, k = ref.bounds(p), val(p.flat(p.q)), val(p.k)
    for r, n in enumerate(p.keys):
        for j in range(n):
            page, row = int(p.bt[r, j // 8]), j % 8
            for hq in range(4):
                s = float(q[r, hq] @ k[page, row, hq // 2])
                assert s <= float(torch.maximum(q[r, hq] * b[page, hq // 2, 0], q[r, hq] * b[page, hq // 2, 1]).sum())


def test_all_pages_is_softmax_attention():
    p = Problem([37], [2], Hq=4, Hkv=2, D=64, DV=64, ps=8, seed=31)
    lists = ref.select(p, e4m3(ref.bounds(p)), 8)
    assert lists[0, 0].tolist() == [0, 1, 2, 3, 4, -1, -1, -1]
    o, lse, mass, _ = ref.attend(p, lists)
    j = torch.arange(37)
    k, v = (val(x)[p.bt[0].long()[j // 8], j % 8] for x in (p.k, p.v))
    for i in range(2):
        for h in range(4):
            n = 36 + i
            z = k[:n, h // 2] @ val(p.q)[0, i, h] / 8.0
            torch.testing.assert_close(o[i, h], torch.softmax(z, 0) @ v[:n, h // 2])
            torch.testing.assert_close(lse[i, h], torch.logsumexp(z, 0))


def test_selection_prefers_high_bounds_and_low_indices():
    p = Problem([80], [1], Hq=1, Hkv=1, D=64, DV=64, ps=8, seed=32)
    b = torch.zeros((p.k.shape[0], 1, 2, 64), dtype=torch.float64)
    p.q = e4m3(torch.ones(1, 1, 1, 64))
    b[int(p.bt[0, 6])] = 1.0
    assert ref.select(p, b, 4)[0, 0].tolist() == [0, 1, 6, 9]
    assert ref.select(p, b, 3, keep_first=0, keep_last=0)[0, 0].tolist() == [0, 1, 6]


def test_rotation_keeps_lengths_and_relative_angles():
    x = torch.randn((1, 1, 64), generator=torch.Generator().manual_seed(3)).double()
    w = fa8.rope_inv_freq(64)
    for inter in (False, True):
        at = lambda n: ref.rope(x, torch.tensor([n]), w, inter, 0, 1.0).flatten()
        assert abs(float(at(5).norm() / x.norm()) - 1) < 1e-12
        assert abs(float(at(5) @ at(9) - at(100) @ at(104))) < 1e-9


def test_expanded_outputs_are_refused():
    """A tensor that a call writes must not have entries that share memory; one that it reads may."""
    assert status(fa8_bounds, BOUNDS, dict(bounds=e8(1, 2, 2, 128).expand(9, 2, 2, 128))) == BAD
    assert status(fa8_select, SELECT, dict(bounds=e8(1, 2, 2, 128).expand(9, 2, 2, 128))) == CUDA
    assert status(fa8_select, SELECT, dict(pages=i32(2, 1, 2, 4).expand(2, 3, 2, 4))) == BAD
    assert status(fa8_fwd, FWD, dict(pages=i32(2, 1, 2, 4).expand(2, 3, 2, 4))) == CUDA
    assert status(fa8_fwd, FWD, dict(out=torch.zeros((2, 3, 1, 128), dtype=torch.bfloat16).expand(2, 3, 8, 128))) == BAD
    assert status(fa8_fwd, FWD, dict(lse=f32(2, 8, 1).expand(2, 8, 3))) == BAD
    assert "lse" in fa8.lib().fa8_last_error().decode()


# ------------------------------------------------------------------ the binding's two ways to pass views
@pytest.fixture(params=["c", "python"])
def entries(request, monkeypatch):
    """The views packed by the CPython module, and by the binding itself."""
    monkeypatch.setattr(fa8, "_entries", {})
    if request.param == "python":
        monkeypatch.setattr(fa8, "_args_module", lambda: None)
    elif fa8._args_module() is None:
        pytest.skip("Python's headers are missing here")


def test_views_reach_the_library(entries):
    assert status(fa8_fwd, FWD, {}) == CUDA
    assert status(fa8_rope, ROPE, dict(rotary_offset=4)) == UNSUPPORTED
    assert "rotary_offset" in fa8.lib().fa8_last_error().decode()
    assert status(fa8_select, SELECT, dict(pages=i32(2, 3, 4, 2).transpose(2, 3))) == BAD
    assert "contiguous" in fa8.lib().fa8_last_error().decode()
    assert status(fa8_bounds, BOUNDS, dict(bounds=e8(9, 3, 2, 128))) == BAD
    assert "Hkv=2, 2, D=128" in fa8.lib().fa8_last_error().decode()
    # strides of more than 32 bits, zero-d tensors
    far = torch.empty_strided((2, 2, 8, 128), (0, 2 ** 33 + 8, 128, 1), dtype=torch.bfloat16, device="meta")
    with pytest.raises((fa8.Fa8Error, RuntimeError)):
        fa8_rope(far, **{k: v for k, v in ROPE.items() if k != "q"})
    assert status(fa8_fwd, FWD, dict(descale_q=torch.tensor(1.0))) == CUDA


def test_views_refuse_what_is_no_tensor(entries):
    with pytest.raises(TypeError, match="dtype"):
        status(fa8_bounds, BOUNDS, dict(cu_seqlens_k=torch.zeros(3, dtype=torch.int64)))
    with pytest.raises(ValueError, match="4 dims"):
        status(fa8_bounds, BOUNDS, dict(bounds=e8(1, 9, 2, 2, 128)))
    with pytest.raises((TypeError, AttributeError)):
        status(fa8_bounds, BOUNDS, dict(cu_seqlens_k="cu"))
    with pytest.raises(OverflowError):
        fa8._entry("fa8_page_bounds")(BOUNDS["k"], BOUNDS["bounds"], None, None, None, 2 ** 70, 0, 0)


OPT_IN = r"""
#include <cstdio>
#include <thread>
#include <chrono>
#include <unistd.h>
#include "fa8_host.h"
static std::atomic<int> limit{0};
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int bytes) {
    usleep(bytes < 1000 ? 60000 : 10000);  // the smaller size takes longer
    limit = bytes;
    return cudaSuccess;
}
static int kernel;
int main() {
    static fa8::host::SmemOptIn opt_in;
    std::thread small([] { opt_in(&kernel, 500, 0); });
    usleep(20000);
    std::thread large([] { opt_in(&kernel, 90000, 0); });
    small.join(), large.join();
    opt_in(&kernel, 80000, 0);
    printf("%d", limit.load());
}
"""


def test_two_threads_opt_in_to_the_larger_shared_memory(tmp_path):
    """A smaller size that is set late must not take back a larger one."""
    src, exe = tmp_path / "opt_in.cpp", tmp_path / "opt_in"
    src.write_text(OPT_IN)
    cuda = os.path.join(os.path.dirname(os.path.realpath(build.nvcc())), "..", "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", cuda, "-I", build.CSRC, "-I",
                    os.path.join(build.ROOT, "include"), str(src), "-o", str(exe)], check=True, capture_output=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout
    assert int(out) == 90000
