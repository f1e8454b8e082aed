"""Refusals and workspaces of attention, block norm and clipping, without a GPU: the library's
argument checks answer before any device work, the torch layer names what it cannot take; and how
sequences are cut into units and starts are held within the rows, run on the host."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "differentiable_rasterizer_gb300", "csrc")


@pytest.fixture(scope="module")
def abi():
    from differentiable_rasterizer_gb300 import abi as A
    from differentiable_rasterizer_gb300 import build
    build.build()
    A.lib()
    return A


ATTENTION = dict(q_rows=40, k_rows=50, sequences=1, q=4096, q_row=256, q_head=64, k=4096, k_row=128, k_head=64, v=4096, v_row=128,
                 v_head=64, q_starts=0, k_starts=0, k_lengths=0, o=4096, o_row=256, o_head=64, lse=0, scale=0.125, heads=4, kv_heads=2,
                 dim=64, type_=1, causal=0, fill=0)
ATTENTION_BWD = dict({k: v for k, v in ATTENTION.items() if k not in ("k_lengths", "o", "o_row", "o_head")}, d_o=4096, do_row=256, do_head=64, lse=4096, dq=4096,
                     dq_row=256, dq_head=64, dk=4096, dk_row=128, dk_head=64, dv=4096, dv_row=128, dv_head=64)
BLOCK_NORM = dict(rows=4, cols=32, h=4096, ldh=32, x=4096, ldx=32, post_weight=4096, gate=4096, ldg=0, weight=4096, s=4096, lds=32, y=4096,
                  ldy=32, y_scale=0, rstd_post=4096, rstd=4096, scale=1.0, eps=1e-6, type_=1, post_type=1, gate_type=1, gate_rows=0,
                  weight_type=1, y_type=1)
BLOCK_NORM_BWD = dict(rows=4, cols=32, dy=4096, lddy=32, ds=0, ldds=0, h=4096, ldh=32, s=4096, lds=32, post_weight=4096, gate=4096, ldg=0,
                      weight=4096, rstd_post=4096, rstd=4096, dh=4096, lddh=32, dx=4096, lddx=32, dgate=4096, lddg=0, dweight=4096,
                      dpost=4096, scale=1.0, type_=1, dy_type=1, post_type=1, gate_type=1, gate_rows=0, weight_type=1)

SIZES = [dict(q_rows=-1), dict(k_rows=-1), dict(q_rows=2 ** 31), dict(sequences=-1), dict(sequences=2), dict(sequences=0), dict(q_starts=4096),
         dict(k_starts=4096), dict(q_starts=4098, k_starts=4096), dict(heads=0), dict(kv_heads=0), dict(kv_heads=3), dict(heads=258, kv_heads=2),
         dict(dim=0), dict(dim=129), dict(type_=0), dict(type_=3), dict(type_=7), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
         dict(scale=float("inf")), dict(q=0), dict(q=4097), dict(q_row=63), dict(q_head=63), dict(k=0), dict(k_row=63), dict(v=0), dict(v_head=63),
         dict(q_row=2 ** 39)]
BAD = {
    "gs_attention": SIZES + [dict(o=0), dict(o_row=128), dict(o_row=64, o_head=64), dict(lse=4098), dict(k_lengths=4098), dict(o=4097)],
    "gs_attention_bwd": SIZES + [dict(lse=0), dict(lse=4098), dict(d_o=0), dict(do_row=63), dict(dq_row=128), dict(dk=0), dict(dv=0),
                                      dict(dk_row=64, dk_head=64), dict(dv_head=63), dict(dq=4097)],
    "gs_block_norm_bwd": [dict(rows=-1), dict(cols=0), dict(cols=16385), dict(type_=3), dict(dy_type=3), dict(dy=0), dict(rstd=0), dict(rstd=4098),
                          dict(weight=0), dict(weight=4097), dict(s=0), dict(lds=31), dict(h=0), dict(ldh=31), dict(rstd_post=0),
                          dict(post_weight=0), dict(post_type=3), dict(gate=0), dict(gate=4097), dict(gate_rows=1), dict(gate_rows=1, ldg=32),
                          dict(dh=4097), dict(lddh=31), dict(lddx=31), dict(ds=4096, ldds=31), dict(dweight=4097), dict(dpost=4097),
                          dict(dgate=4097), dict(scale=float("nan")), dict(dy=0, weight=0, rstd=0, dweight=0)],
}
BASE = {"gs_attention": ATTENTION, "gs_attention_bwd": ATTENTION_BWD, "gs_block_norm_bwd": BLOCK_NORM_BWD}


def pack(abi, name, args):
    return getattr(abi, name[3:] + "_args")(**args)


@pytest.mark.parametrize("name", sorted(BAD))
def test_bad_arguments(abi, name):
    """Refused with a workspace of any size, before device work."""
    for change in BAD[name]:
        args = pack(abi, name, dict(BASE[name], **change))
        assert getattr(abi.lib(), name)(args, 4096, ctypes.byref(ctypes.c_size_t(1 << 40)), None) == abi.GS_ERR_INVALID_ARG, change
    assert getattr(abi.lib(), name)(None, None, None, None) == abi.GS_ERR_INVALID_ARG


def test_bad_block_norm_arguments(abi):
    for change in (dict(rows=-1), dict(cols=0), dict(cols=16385), dict(h=0), dict(ldh=31), dict(x=0), dict(ldx=31), dict(s=0), dict(lds=31),
                   dict(y=0), dict(ldy=31), dict(type_=3), dict(post_type=3), dict(weight_type=3), dict(gate_type=3), dict(y_type=4),
                   dict(y_type=3), dict(y_scale=4096), dict(weight=0), dict(weight=0, rstd=0), dict(post_weight=0), dict(gate_rows=1),
                   dict(gate_rows=1, gate=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(h=4097), dict(rstd=4098), dict(rstd_post=4097)):
        with pytest.raises(abi.GsError) as e:
            abi.gs_block_norm(**dict(BLOCK_NORM, **change), stream=None)
        assert e.value.status == abi.GS_ERR_INVALID_ARG, change


def clip(abi, tensors, norm=4096, max_norm=1.0, ws=4096, size=1 << 40):
    args, table = abi.clip_norm_args(tensors, norm, max_norm)
    n = ctypes.c_size_t(size)
    status = abi.lib().gs_clip_norm(args, ws, ctypes.byref(n), None)
    del table
    return status, n.value


def test_bad_clip_arguments(abi):
    a, b = (65536, 65536, 100, 0, 0), (131072, 196608, 100, 1, 0)
    for tensors in ([(0, 65536, 1, 0, 0)], [(65536, 0, 1, 0, 0)], [(65537, 65536, 1, 0, 0)], [(65536, 131074, 1, 0, 0)], [(65536, 65536, -1, 0, 0)],
                    [(65536, 131072, 1, 3, 0)], [(65536, 131072, 1, 0, 3)], [(65536, 65536, 4, 0, 1)], [a, a], [a, (65536 + 396, 65536 + 396, 1, 0, 0)],
                    [(65536, 65536 + 200, 100, 0, 0)], [b, (131072, 262144, 1, 1, 1)], [b, (262144, 196608, 1, 0, 0)], [(65536, 65536, 2 ** 45, 0, 0)]):
        assert clip(abi, tensors)[0] == abi.GS_ERR_INVALID_ARG, tensors
    assert clip(abi, [a] * 1025)[0] == abi.GS_ERR_INVALID_ARG
    assert clip(abi, [a], max_norm=-1.0)[0] == clip(abi, [a], max_norm=float("nan"))[0] == abi.GS_ERR_INVALID_ARG
    assert clip(abi, [a], norm=0)[0] == clip(abi, [a], norm=4098)[0] == abi.GS_ERR_INVALID_ARG
    assert clip(abi, [a], size=8)[0] == clip(abi, [a], ws=4096 + 16)[0] == abi.GS_ERR_INVALID_ARG
    ok, need = clip(abi, [a, b, (65536 + 400, 65536 + 400, 5, 0, 0), (0, 0, 0, 0, 0)], ws=None)   # neighbours, an empty one
    assert ok == abi.GS_OK and need > 0 and need % 256 == 0


def test_workspaces(abi):
    """Queries answer without device work; too small, misaligned or missing scratch is refused."""
    one = dict(ATTENTION, q_rows=1, k_rows=100000)           # parts of the keys
    odd = dict(ATTENTION, q=4098)                            # a copy of q
    for name, base in (("gs_attention", one), ("gs_attention", odd), ("gs_attention_bwd", ATTENTION_BWD),
                       ("gs_block_norm_bwd", BLOCK_NORM_BWD)):
        args = pack(abi, name, base)
        need = abi.layer_ws_bytes(name, args)
        assert need > 0 and need % 256 == 0, name
        f = getattr(abi.lib(), name)
        for ws, size in ((4096, need - 1), (4096 + 16, need), (4096, 0)):
            assert f(args, ws, ctypes.byref(ctypes.c_size_t(size)), None) == abi.GS_ERR_INVALID_ARG, (name, ws, size)
        assert f(args, None, None, None) == abi.GS_ERR_INVALID_ARG
    # scratch goes with the rows of queries, whatever the keys
    a, b = (abi.layer_ws_bytes("gs_attention", pack(abi, "gs_attention", dict(one, k_rows=n))) for n in (10 ** 6, 10 ** 9))
    assert a < 2 ** 20 and b < 2 ** 20


def test_calls_that_need_no_device(abi):
    assert abi.gs_attention(pack(abi, "gs_attention", dict(ATTENTION, q_rows=0, q=0, o=0)), None, None, None) is None
    nothing = dict(ATTENTION_BWD, q_rows=0, k_rows=0, q=0, k=0, v=0, d_o=0, lse=0)
    need = abi.layer_ws_bytes("gs_attention_bwd", pack(abi, "gs_attention_bwd", nothing))
    assert abi.gs_attention_bwd(pack(abi, "gs_attention_bwd", nothing), 4096, need, None) is None
    abi.gs_block_norm(**dict(BLOCK_NORM, rows=0, h=0, x=0, s=0, y=0), stream=None)
    none = dict(BLOCK_NORM_BWD, rows=0, dweight=0, dpost=0, dgate=0)
    assert abi.gs_block_norm_bwd(pack(abi, "gs_block_norm_bwd", none), None, None, None) is None
    for call, name, base in ((abi.gs_attention, "gs_attention", ATTENTION), (abi.gs_attention_bwd, "gs_attention_bwd", ATTENTION_BWD),
                             (abi.gs_block_norm_bwd, "gs_block_norm_bwd", BLOCK_NORM_BWD)):
        with pytest.raises(abi.GsError) as e:
            call(pack(abi, name, dict(base, **({"rows": -1} if "rows" in base else {"q_rows": -1}))), None, None, None)
        assert e.value.status == abi.GS_ERR_INVALID_ARG
    args, table = abi.clip_norm_args([], 0, 1.0)
    with pytest.raises(abi.GsError):
        abi.gs_clip_norm(args, 4096, 1 << 20, None)


def test_tensor_refusals(abi):
    from differentiable_rasterizer_gb300 import layers
    q, h = torch.zeros((4, 2, 8), dtype=torch.bfloat16), torch.zeros((4, 8))
    for call in (lambda: layers.attention(q, q, q), lambda: layers.attention_backward(q, q, q, q, q, h), lambda: layers.block_norm(h, h, h[0]),
                 lambda: layers.block_norm_backward(h, h, h, h[0], h[:, 0]), lambda: layers.clip_norm([h], 1.0)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    for call, match in ((lambda: layers.attention(None, q, q), "q: expected a tensor"), (lambda: layers.clip_norm([], 1.0), "tensors: 1 to"),
                        (lambda: layers.clip_norm(h, 1.0), "expected a list"), (lambda: layers.clip_norm([h], 1.0, out=[]), "out: expected"),
                        (lambda: layers.block_norm([1.0], h), "h: expected a tensor")):
        with pytest.raises(ValueError, match=match):
            call()


PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "attention.cuh"

using namespace gs::attn;

int main()
{
    int wrong = 0;
    const int64_t big = 0x7fffffff;
    wrong += held(-5, 0, 10) != 0 || held(11, 0, 10) != 10 || held(7, 0, 10) != 7 || held(big, 3, 3) != 3 || held(-big, 3, 9) != 3;
    // units of every cut of some rows into sequences are within the bound that the grid is made for
    std::srand(1);
    for (int trial = 0; trial < 20000; ++trial) {
        const int n = std::rand() % 40, tokens = 1 + std::rand() % 130;
        int64_t rows = 0, units = 0;
        for (int s = 0; s < n; ++s) {
            const int len = std::rand() % 3 ? std::rand() % 400 : std::rand() % 2;
            rows += len;
            units += (len + tokens - 1) / tokens;
        }
        rows += std::rand() % 3 * 100;   // rows of no sequence
        wrong += units > units_at_most(rows, n, true, tokens);
        wrong += units_at_most(rows, 1, false, tokens) < (rows + tokens - 1) / tokens;
    }
    // keys that a query sees, against their definition
    for (int lq = 0; lq < 6; ++lq)
        for (int lk = 0; lk < 6; ++lk)
            for (int i = 0; i < lq; ++i) {
                int seen = 0;
                for (int j = 0; j < lk; ++j) seen += j <= i + lk - lq;
                const Sequence s = {0, lq, 0, lk};
                wrong += keys_seen(s, i, true) != seen || keys_seen(s, i, false) != lk;
            }
    std::printf("%d\n", wrong);
    return wrong != 0;
}
"""


def test_units_and_starts_on_the_host(tmp_path):
    from differentiable_rasterizer_gb300 import build
    src, out = tmp_path / "units.cu", tmp_path / "units"
    src.write_text(PROGRAM)
    subprocess.run([build._nvcc(), "-std=c++17", "--extended-lambda", "-I", CSRC, *build.ARCH, str(src), "-o", str(out)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("name,rings,blocks", [("attention.cu", 1, 1), ("attention_bwd.cu", 5, 2)])
def test_blocks_end_after_their_copies_and_products(name, rings, blocks):
    """Each producer ends with a wait for its last copies, each issuing lane with one for its products, blind to the block's flag."""
    text = open(os.path.join(CSRC, name)).read()
    assert len(re.findall(r"last_copies<[\w:]+>\(.*mbar_wait_alone\(", text)) == rings
    assert len(re.findall(r"mma_commit<false>\(bars \+ 8 \* \(S::kDone \+ \w+\)\);[^\n]*\n\s*if \(!mbar_wait_alone\(", text)) == blocks
