"""Host-side checks of the C ABI in include/fp8mm_block.h (no GPU): every symbol is
exported and bound, queries answer, and bad arguments are refused before any launch.
Every call below fails a check or has nothing to do, so nothing is ever enqueued (the
fake non-null pointers are never dereferenced)."""

import os
import re
import shutil
import subprocess

import pytest
import torch

import precision_matmul_amd as fp8mm
from precision_matmul_amd import _lib, block, moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8mm_block.h")
FAKE = 0x1000
NAN, INF = float("nan"), float("inf")
EINVAL, ENOTIMPL, OK = _lib.EINVAL, _lib.ENOTIMPL, _lib.OK


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libfp8mm.so is not built (run __graft_entry__.build())")
    return _lib.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fp8_\w+|fp8mm_\w+)\s*\(", text)))
    assert len(names) == 10, names
    for n in names:
        assert hasattr(lib, n) and n in _lib.SIGNATURES, n


CALLS = {
    "fp8mm_rms_norm": dict(x=FAKE, ldx=256, res=FAKE, ldr=256, dt=0, R=4, C=256, w=FAKE, pd=0, eps=1e-6, h=FAKE,
                           ldh=256, y=FAKE, ldy=256, q=FAKE, ldq=256, s=FAKE, recipe=2, rstd=FAKE, st=None),
    "fp8mm_rms_norm_backward": dict(dy=FAKE, lddy=64, h=FAKE, ldh=64, gh=FAKE, ldg=64, dt=0, R=4, C=64, w=None, pd=0,
                                    rstd=FAKE, dx=FAKE, lddx=64, dw=FAKE, ws=FAKE, wsb=1 << 20, st=None),
    "fp8mm_moe_balance_loss": dict(l=FAKE, dt=0, T=16, E=64, ld=64, ids=FAKE, k=6, score=0, ends=FAKE, S=3, coeff=1.0,
                                   loss=FAKE, counts=FAKE, tokens=FAKE, ws=FAKE, wsb=1 << 20, st=None),
    "fp8mm_moe_balance_loss_backward": dict(g=FAKE, l=FAKE, dt=0, T=16, E=64, ld=64, counts=FAKE, tokens=FAKE, k=6,
                                            score=0, ends=FAKE, S=3, coeff=1.0, out=FAKE, ldg=64, st=None),
    "fp8mm_lora": dict(x=FAKE, ldx=64, T=8, K=64, down=FAKE, up=FAKE, n=4, r=16, N=96, ids=FAKE, scales=None,
                       base=FAKE, ldb=96, out=FAKE + 64, ldo=96, v=FAKE, st=None),
    "fp8mm_lora_backward": dict(dy=FAKE, lddy=96, x=FAKE, ldx=64, T=8, K=64, down=FAKE, up=FAKE, n=4, r=16, N=96,
                                ids=FAKE, scales=None, v=FAKE, dx=FAKE, lddx=64, ddown=FAKE, dup=FAKE, gd=0, ws=FAKE,
                                wsb=1 << 24, st=None),
}


def _call(lib, name, kw):
    a = dict(CALLS[name])
    assert set(kw) <= set(a), kw
    a.update(kw)
    return getattr(lib, name)(*a.values())


@pytest.mark.parametrize("name,kw,code", [(n, kw, c) for n, cases in {
    "fp8mm_rms_norm": [
        (dict(dt=2), EINVAL), (dict(pd=7), EINVAL), (dict(R=-1), EINVAL), (dict(C=0), EINVAL), (dict(R=2 ** 31), EINVAL),
        (dict(C=2 ** 22 + 128, ldx=2 ** 23, ldr=2 ** 23, ldh=2 ** 23, ldy=2 ** 23, ldq=2 ** 23), EINVAL),
        (dict(ldx=255), EINVAL), (dict(ldr=255), EINVAL), (dict(ldh=255), EINVAL), (dict(ldy=255), EINVAL),
        (dict(ldq=255), EINVAL), (dict(ldq=264), EINVAL), (dict(ldx=2 ** 40 + 1), EINVAL),
        (dict(eps=-1.0), EINVAL), (dict(eps=NAN), EINVAL), (dict(eps=INF), EINVAL), (dict(x=None), EINVAL),
        (dict(s=None), EINVAL), (dict(x=FAKE + 1), EINVAL), (dict(res=FAKE + 1), EINVAL), (dict(h=FAKE + 1), EINVAL),
        (dict(y=FAKE + 1), EINVAL), (dict(q=FAKE + 8), EINVAL), (dict(s=FAKE + 2), EINVAL), (dict(rstd=FAKE + 2), EINVAL),
        (dict(pd=1, w=FAKE + 2), EINVAL), (dict(C=192, recipe=2), EINVAL), (dict(C=200, recipe=1), EINVAL),
        (dict(recipe=0), ENOTIMPL), (dict(recipe=3), ENOTIMPL), (dict(recipe=5), ENOTIMPL), (dict(recipe=9), EINVAL),
        (dict(dt=1), ENOTIMPL), (dict(dt=1, q=None, x=FAKE + 2), EINVAL)],
    "fp8mm_rms_norm_backward": [
        (dict(lddy=10), EINVAL), (dict(ldh=10), EINVAL), (dict(ldg=10), EINVAL), (dict(lddx=10), EINVAL),
        (dict(dy=None), EINVAL), (dict(h=None), EINVAL), (dict(rstd=None), EINVAL), (dict(R=9000, ws=None), EINVAL),
        (dict(R=9000, wsb=64), EINVAL), (dict(R=9000, ws=FAKE + 4), EINVAL), (dict(dt=3), EINVAL), (dict(C=-1), EINVAL),
        (dict(dw=FAKE + 1), EINVAL), (dict(dx=FAKE + 1), EINVAL), (dict(gh=FAKE + 1), EINVAL),
        (dict(dx=FAKE, gh=FAKE, lddx=128), EINVAL)],
    "fp8mm_moe_balance_loss": [
        (dict(dt=2), EINVAL), (dict(score=2), EINVAL), (dict(T=-1), EINVAL), (dict(E=0), EINVAL), (dict(S=0), EINVAL),
        (dict(S=2 ** 20 + 1), EINVAL), (dict(ends=None), EINVAL), (dict(k=0), EINVAL), (dict(T=2 ** 30), EINVAL),
        (dict(coeff=NAN), EINVAL), (dict(coeff=INF), EINVAL), (dict(ld=63), EINVAL), (dict(l=None), EINVAL),
        (dict(ids=None), EINVAL), (dict(loss=None), EINVAL), (dict(counts=None), EINVAL), (dict(tokens=None), EINVAL),
        (dict(l=FAKE + 1), EINVAL), (dict(ws=None), EINVAL), (dict(wsb=8), EINVAL), (dict(T=2000, wsb=100), EINVAL), (dict(ws=FAKE + 8), EINVAL),
        (dict(E=1025, ld=1025), ENOTIMPL), (dict(k=65), ENOTIMPL), (dict(E=4096, ld=4096, S=2 ** 19), EINVAL)],
    "fp8mm_moe_balance_loss_backward": [
        (dict(g=None), EINVAL), (dict(l=None), EINVAL), (dict(counts=None), EINVAL), (dict(tokens=None), EINVAL),
        (dict(out=None), EINVAL), (dict(ldg=63), EINVAL), (dict(ld=63), EINVAL), (dict(k=0), EINVAL),
        (dict(score=-1), EINVAL), (dict(out=FAKE + 1), EINVAL), (dict(ends=None), EINVAL), (dict(coeff=NAN), EINVAL),
        (dict(E=1025, ld=1025, ldg=1025), ENOTIMPL)],
    "fp8mm_lora": [
        (dict(T=-1), EINVAL), (dict(T=2 ** 31), EINVAL), (dict(n=0), EINVAL), (dict(n=2 ** 31), EINVAL),
        (dict(r=0), EINVAL), (dict(r=257), ENOTIMPL), (dict(K=0), EINVAL), (dict(N=0), EINVAL),
        (dict(K=2 ** 22 + 1, ldx=2 ** 23), EINVAL), (dict(N=2 ** 22 + 1, ldb=2 ** 23, ldo=2 ** 23), EINVAL),
        (dict(ldx=63), EINVAL), (dict(ldb=95), EINVAL), (dict(ldo=95), EINVAL), (dict(x=None), EINVAL),
        (dict(down=None), EINVAL), (dict(up=None), EINVAL), (dict(ids=None), EINVAL), (dict(out=None), EINVAL),
        (dict(v=None), EINVAL), (dict(x=FAKE + 1), EINVAL), (dict(up=FAKE + 1), EINVAL), (dict(v=FAKE + 2), EINVAL),
        (dict(scales=FAKE + 2), EINVAL), (dict(out=FAKE, ldb=128), EINVAL),
        (dict(T=2 ** 30, N=2 ** 14, ldb=2 ** 14, ldo=2 ** 14), EINVAL)],
    "fp8mm_lora_backward": [
        (dict(gd=2), EINVAL), (dict(lddy=95), EINVAL), (dict(ldx=63), EINVAL), (dict(lddx=63), EINVAL),
        (dict(dy=None), EINVAL), (dict(x=None), EINVAL), (dict(v=None), EINVAL), (dict(ids=None), EINVAL),
        (dict(ws=None), EINVAL), (dict(wsb=64), EINVAL), (dict(ws=FAKE + 8), EINVAL), (dict(r=257), ENOTIMPL),
        (dict(gd=1, dup=FAKE + 2), EINVAL), (dict(dx=FAKE + 1), EINVAL), (dict(n=1025), ENOTIMPL)],
}.items() for kw, c in cases])
def test_refusals(lib, name, kw, code):
    assert _call(lib, name, kw) == code
    assert lib.fp8mm_last_error().decode()


@pytest.mark.parametrize("name,kw", [
    ("fp8mm_rms_norm", dict(R=0, x=None, s=None)),
    ("fp8mm_rms_norm", dict(res=None, y=None, q=None, rstd=None)),
    ("fp8mm_rms_norm_backward", dict(dx=None, dw=None)),
    ("fp8mm_rms_norm_backward", dict(R=0, dy=None, h=None, rstd=None, dw=None)),
    ("fp8mm_moe_balance_loss_backward", dict(T=0, l=None)),
    ("fp8mm_lora", dict(T=0, x=None, ids=None, v=None)),
    ("fp8mm_lora_backward", dict(T=0, ddown=None, dup=None, ids=None, dy=None)),
    ("fp8mm_lora_backward", dict(dx=None, ddown=None, dup=None)),
])
def test_calls_with_nothing_to_do(lib, name, kw):
    assert _call(lib, name, kw) == OK


def test_queries(lib):
    assert lib.fp8mm_rms_norm_backward_workspace(4, 64) == 0            # one launch, nothing kept between
    assert 0 < lib.fp8mm_rms_norm_backward_workspace(9000, 64) <= 1 << 20
    assert lib.fp8mm_rms_norm_backward_workspace(-1, 64) == -1
    assert 0 < lib.fp8mm_rms_norm_backward_workspace(2 ** 30, 64) <= 4096 * 64 * 4     # bounded in the rows
    assert lib.fp8mm_moe_balance_loss_workspace(16384, 64, 1) > 0
    assert lib.fp8mm_moe_balance_loss_workspace(16, 64, 1) == 0         # one workgroup
    assert 0 < lib.fp8mm_moe_balance_loss_workspace(16, 64, 2)
    assert lib.fp8mm_moe_balance_loss_workspace(0, 64, 1) == 0
    assert lib.fp8mm_moe_balance_loss_workspace(16, 64, 0) == -1
    assert lib.fp8mm_moe_balance_loss_workspace(2 ** 31 - 1, 64, 1) < 1 << 20          # bounded in the tokens
    for bad in ((-1, 64, 4, 16), (8, 0, 4, 16), (8, 64, 0, 16), (8, 64, 4, 0), (8, 64, 4, 257)):
        assert lib.fp8mm_lora_splits(*bad) == -1
    for T in (0, 1, 16, 300, 5000, 10 ** 6):
        assert 1 <= lib.fp8mm_lora_splits(T, 5120, 8, 16) <= 16
    assert lib.fp8mm_lora_splits(8, 64, 8, 16) == 1                     # nothing to split
    assert lib.fp8mm_lora_backward_workspace(8, 64, 64, 4, 16) >= 4 * 8 * 16
    assert lib.fp8mm_lora_backward_workspace(8, 64, 0, 4, 16) == -1


def test_binding_refuses_what_is_not_on_a_device():
    x, ids = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros((4, 2), dtype=torch.int32)
    panels = torch.zeros((2, 16, 128), dtype=torch.bfloat16)
    for call in (lambda: fp8mm.rms_norm_forward(x), lambda: fp8mm.fp8_rms_norm_forward(x),
                 lambda: fp8mm.rms_norm_backward(x, x, None, x[:, 0].float()), lambda: fp8mm.rms_norm(x),
                 lambda: fp8mm.moe_balance_loss_forward(x, ids), lambda: fp8mm.moe_balance_loss(x, ids),
                 lambda: fp8mm.lora_forward(x, panels, panels, ids[:, 0].contiguous()),
                 lambda: fp8mm.lora(x, panels, panels, ids[:, 0])):
        with pytest.raises(ValueError):
            call()


def test_header_compiles_as_c99_and_links(lib, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no gcc")
    src = tmp_path / "block.c"
    src.write_text(r"""
#include <stdio.h>
#include <string.h>
#include "fp8mm_block.h"
int main(void) {
  if (fp8mm_rms_norm_backward_workspace(4, 64) != 0 || fp8mm_lora_splits(-1, 6, 64, 1) != -1) return 1;
  fp8mm_status st = fp8mm_moe_balance_loss(0, FP8MM_OUT_BF16, 4, 64, 64, 0, 65, FP8MM_SCORE_SIGMOID, 0, 1, 1.0f, 0, 0, 0,
                                           0, 0, 0);
  if (st != FP8MM_ENOTIMPL || strlen(fp8mm_last_error()) == 0) return 2;
  if (fp8mm_lora(0, 64, 0, 64, 0, 0, 1, 8, 64, 0, 0, 0, 64, 0, 64, 0, 0) != FP8MM_OK) return 3;
  printf("ok\n");
  return 0;
}
""")
    exe = tmp_path / "block"
    libdir = os.path.dirname(_lib.LIB_PATH)
    cmd = [gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", f"-I{os.path.join(ROOT, 'include')}",
           "-I/opt/rocm/include", str(src), f"-L{libdir}", "-lfp8mm", f"-Wl,-rpath,{libdir}", "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and run.stdout.strip() == "ok", (run.returncode, run.stdout, run.stderr)


def _on_the_host(monkeypatch):
    """The library's calls behind lora, fp8_swiglu and fp8_moe replaced by ones that check
    nothing and compute zeros, so that their Python paths run on CPU tensors."""
    monkeypatch.setattr(block, "lora_forward", lambda x, down, up, ids, scales=None, base=None: (
        x.new_zeros((x.shape[0], up.shape[2])), torch.zeros(1, x.shape[0], down.shape[1])))
    monkeypatch.setattr(moe, "fp8_swiglu_forward", lambda x, recipe, checkpoint: (
        x.new_zeros((x.shape[0], x.shape[1] // 2)), (x, x) if checkpoint else None))
    monkeypatch.setattr(moe, "_experts_forward", lambda x, *rest: (torch.zeros_like(x), ()))


def _lora_inputs():
    return (torch.zeros((4, 16), dtype=torch.bfloat16), torch.zeros((2, 8, 16), dtype=torch.bfloat16),
            torch.zeros((2, 8, 32), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), torch.ones(2),
            torch.zeros((4, 32), dtype=torch.bfloat16))


@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_derivatives_are_refused_not_dropped(monkeypatch, grad):
    """A dual tensor has no requires_grad: its tangent must not vanish on the way."""
    _on_the_host(monkeypatch)
    ad = torch.autograd.forward_ad
    rows, panel = torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros((2, 256, 256), dtype=torch.bfloat16)
    ids, weights = torch.zeros((4, 1), dtype=torch.int32), torch.ones((4, 1))
    calls = [(fp8mm.lora, _lora_inputs(), (0, 1, 2, 4, 5)), (fp8mm.fp8_swiglu, (rows,), (0,)),
             (fp8mm.fp8_moe, (rows, panel, panel, ids, weights), (0, 1, 2, 4))]
    with torch.set_grad_enabled(grad):
        for fn, args, moved in calls:
            fn(*args)                    # without a tangent: runs, inside a dual level too
            for i in moved:
                with ad.dual_level():
                    fn(*args)
                    duals = [ad.make_dual(t, torch.ones_like(t)) if j == i else t for j, t in enumerate(args)]
                    with pytest.raises(NotImplementedError):
                        fn(*duals)


def test_a_gradient_of_the_scales_is_refused(monkeypatch):
    """There is none: asked for, it must not be missing without a word."""
    _on_the_host(monkeypatch)
    x, down, up, ids, scales, base = _lora_inputs()
    needs = scales.clone().requires_grad_()
    for leaf in (x, x.clone().requires_grad_()):
        with pytest.raises(NotImplementedError):
            fp8mm.lora(leaf, down, up, ids, needs, base)
        assert fp8mm.lora(leaf, down, up, ids, needs.detach(), base).requires_grad == leaf.requires_grad
    with torch.no_grad():
        assert not fp8mm.lora(x.clone().requires_grad_(), down, up, ids, needs, base).requires_grad


@pytest.mark.parametrize("grad", [True, False])
def test_lora_makes_its_inputs_dense_with_and_without_a_gradient(monkeypatch, grad):
    """Transposed matrices, spread ids and scales: what trains runs without a gradient too."""
    def forward(*args):
        assert all(t is None or t.is_contiguous() for t in args)
        return torch.zeros((4, 32), dtype=torch.bfloat16), torch.zeros(1, 4, 8)

    monkeypatch.setattr(block, "lora_forward", forward)
    x, down, up, ids, scales, base = _lora_inputs()

    def spread(t):
        wide = t.new_zeros((*t.shape[::-1], 2))[..., 0].permute(*range(t.dim())[::-1])
        assert wide.shape == t.shape and not wide.is_contiguous()
        return wide.requires_grad_(grad and t.dtype == torch.bfloat16)

    for args in ((x, down, up, ids, scales, base), (x, down, up, ids, None, None)):
        out = fp8mm.lora(*(None if t is None else spread(t) for t in args))
        assert out.requires_grad == grad


def test_any_finite_eps_is_accepted(lib):
    """Of both norms: what the headers say."""
    from tests import test_host_abi_moe as abi

    for eps, code in ((0.0, OK), (1.0000001e30, OK), (3.4028234e38, OK), (-1e-45, EINVAL), (INF, EINVAL), (NAN, EINVAL)):
        assert _call(lib, "fp8mm_rms_norm", dict(R=0, x=None, s=None, eps=eps)) == code, eps
        assert abi._call(lib, "fp8mm_layer_norm", abi.NORM, abi.NORM_D, dict(R=0, x=None, y=None, eps=eps)) == code, eps
