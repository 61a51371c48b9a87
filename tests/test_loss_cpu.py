"""The loss operators' C ABI and binding without a GPU: every declared name is
exported and bound, and bad arguments come back as errors before anything is
enqueued (the addresses below are never touched)."""
import ctypes as C
import os
import re
import subprocess

import pytest
import torch

import gradient_all_reduce_worker_amd as pkg
from gradient_all_reduce_worker_amd import _loss, _native

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL = -1
NAN, INF = float("nan"), float("inf")


def _declared():
    text = open(os.path.join(ROOT, "include", "ga_loss.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(ga_[a-z0-9_]+)\s*\(", text)))


def test_declared_exported_and_bound():
    names = _declared()
    assert set(names) == set(_loss.LOSS_EXPORTS)
    syms = subprocess.run(["nm", "-D", "--defined-only", _native.LIB_PATH], capture_output=True, text=True,
                          check=True).stdout
    exported = {line.split()[-1] for line in syms.splitlines() if " T " in line}
    assert set(names) <= exported
    assert all(callable(getattr(pkg, n)) for n in names)


def _ptrs(*vals):
    return (C.c_void_p * len(vals))(*vals)


def _tok(*vals):
    return (C.c_int64 * len(vals))(*vals)


X, G = _ptrs(0x100000, 0x200000), _ptrs(0x300000, 0x400000)
I, V, W, R = (_ptrs(b, b + 0x8000) for b in (0x500000, 0x600000, 0x700000, 0x800000))
T2 = _tok(3, 5)
WS, OUT, CNT = 0x900000, 0xA00000, 0xB00000


def _distill(**k):
    a = dict(logits=X, tokens=T2, P=2, V=40, ld=40, dt=0, idx=I, vals=V, vdt=0, lse=W, K=4, weight=None, temp=1.0,
             scale=1.0, grad=G, ldg=40, row=R, out=OUT, ws=WS, ws_bytes=1 << 20, stream=None)
    a.update(k)
    return _loss.load().ga_distill_loss(*a.values())


def _top(**k):
    a = dict(logits=X, tokens=T2, P=2, V=40, ld=40, dt=0, K=4, temp=1.0, vals=V, idx=I, lse=W, stream=None)
    a.update(k)
    return _loss.load().ga_top_logits(*a.values())


def _balance(**k):
    a = dict(logits=X, tokens=T2, P=2, E=40, ld=40, dt=0, idx=I, K=4, mask=W, score=0, group=0, scale=1.0, grad=G,
             ldg=40, counts=CNT, out=OUT, ws=WS, ws_bytes=1 << 20, stream=None)
    a.update(k)
    return _loss.load().ga_balance_loss(*a.values())


COMMON = [dict(P=0), dict(P=65), dict(tokens=None), dict(tokens=_tok(3, -1)), dict(tokens=_tok(1 << 31, 0)),
          dict(tokens=_tok((1 << 31) - 1, 1)), dict(dt=2), dict(dt=-1), dict(ld=39), dict(K=0), dict(K=1025),
          dict(logits=None), dict(logits=_ptrs(0x100000, 0)), dict(logits=_ptrs(0x100002, 0x200000)),
          dict(idx=None), dict(idx=_ptrs(0, 0x508000)), dict(idx=_ptrs(0x500002, 0x508000)),
          dict(ld=1 << 62), dict(ld=1 << 46)]


@pytest.mark.parametrize("bad", COMMON + [
    dict(V=0), dict(V=1 << 31), dict(K=41), dict(temp=0.0), dict(temp=-1.0), dict(temp=NAN), dict(temp=INF),
    dict(temp=1e-44), dict(vals=None), dict(vals=_ptrs(0x600002, 0x608000)), dict(lse=_ptrs(0x700001, 0x708000)),
    dict(vals=_ptrs(0x100000 + 4 * 119, 0x608000)),                       # inside worker 0's logits
    dict(idx=_ptrs(0x500000, 0x500020)),                                  # the workers' outputs overlap
    dict(lse=_ptrs(0x600000, 0x708000))])                                 # on vals
def test_top_refusals(bad):
    assert _top(**bad) == EINVAL
    assert b"ga_top_logits" in _native.load().ga_last_error()


@pytest.mark.parametrize("bad", COMMON + [
    dict(V=0), dict(V=1 << 31), dict(temp=0.0), dict(temp=NAN), dict(temp=INF), dict(temp=1e-44), dict(scale=NAN),
    dict(scale=INF), dict(vdt=7), dict(vals=None), dict(vals=_ptrs(0x600002, 0x608000)), dict(out=None),
    dict(out=OUT + 2), dict(ws=None), dict(ws=WS + 4), dict(ws_bytes=8), dict(ldg=39),
    dict(grad=_ptrs(0x300002, 0x400000)), dict(grad=_ptrs(0, 0x400000)),
    dict(grad=X, ldg=44),                                                 # in place with another stride
    dict(grad=_ptrs(0x100000 + 4, 0x400000)),                             # half on the logits
    dict(grad=_ptrs(0x100000, 0x400000)),                                 # one worker in place, one not
    dict(grad=_ptrs(0x200000, 0x100000)),                                 # another worker's logits
    dict(grad=_ptrs(0x300000, 0x300000 + 4)), dict(row=_ptrs(0x300000, 0x808000)), dict(row=_ptrs(0x800002, 0x808000)),
    dict(weight=_ptrs(0x900001, 0x908000)), dict(weight=W, row=W), dict(out=WS), dict(out=0x500000)])
def test_distill_refusals(bad):
    assert _distill(**bad) == EINVAL
    assert b"ga_distill_loss" in _native.load().ga_last_error()


@pytest.mark.parametrize("temp", [2.9387359e-39, 3e-39, 4e-39, 4.2e-39])
def test_temperatures_below_the_kernels_range(temp):
    """1 / temp is finite there, log2(e) / temp is not."""
    assert _top(temp=temp) == EINVAL and b"temp" in _native.load().ga_last_error()
    assert _distill(temp=temp) == EINVAL and b"temp" in _native.load().ga_last_error()


@pytest.mark.parametrize("bad", COMMON + [
    dict(E=0), dict(E=1025, ld=1025, ldg=1025), dict(score=2), dict(score=-1), dict(group=-1), dict(scale=NAN),
    dict(counts=None), dict(counts=CNT + 2), dict(out=None), dict(ws=None), dict(ws=WS + 4), dict(ws_bytes=8),
    dict(mask=_ptrs(0, 0x708000)), dict(ldg=39), dict(grad=X, ldg=44), dict(grad=_ptrs(0x100000, 0x400000)),
    dict(counts=0x300000), dict(counts=0x500000), dict(out=WS + 8),
    dict(tokens=_tok(1 << 30, 1), K=4, ld=40)])
def test_balance_refusals(bad):
    assert _balance(**bad) == EINVAL
    assert b"ga_balance_loss" in _native.load().ga_last_error()


def test_groups_and_workspace_sizes():
    assert pkg.ga_balance_groups([5, 0, 9], 0) == 1
    assert pkg.ga_balance_groups([5, 0, 9], 4) == 2 + 0 + 3
    assert pkg.ga_balance_groups([5], 1 << 40) == 1
    assert _loss.load().ga_balance_groups(_tok(-1), 1, 0) == 0
    assert pkg.ga_balance_loss_ws_bytes([5, 0, 9], 16, 4) > 0
    assert pkg.ga_balance_loss_ws_bytes([5], 0) == 0 and pkg.ga_balance_loss_ws_bytes([5], 1025) == 0
    assert pkg.ga_distill_loss_ws_bytes(0) == 0 and pkg.ga_distill_loss_ws_bytes(7) % 8 == 0
    # every size of the workspace keeps the parts aligned
    for rows in (1, 63, 64, 65, 4097, 1 << 20):
        for E in (1, 7, 64, 1024):
            assert pkg.ga_balance_loss_ws_bytes([rows, 3], E, 0) >= 8


def test_no_rows_is_a_success_for_top():
    assert _top(tokens=_tok(0, 0), logits=_ptrs(0, 0), idx=_ptrs(0, 0), vals=_ptrs(0, 0), lse=None) == 0


def test_binding_refuses_before_the_library():
    z = [torch.zeros(2, 8)]
    i = [torch.zeros(2, 3, dtype=torch.int32)]
    for f in (lambda: pkg.ga_top_logits(z, 3), lambda: pkg.ga_distill_loss(z, i, [torch.zeros(2, 3)]),
              lambda: pkg.ga_balance_loss(z, i), lambda: pkg.ga_top_logits([], 3)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        pkg.ga_top_logits([torch.zeros(2, 8, dtype=torch.float16)], 3)


def test_the_library_is_linked_without_the_binding(tmp_path, monkeypatch):
    """Where the binding's module cannot be built (no host compiler, no torch
    headers) libga.so is there all the same, and the failure is reported."""
    from gradient_all_reduce_worker_amd import build

    linker = tmp_path / "hipcc"
    linker.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho linked > "$2"\n')
    linker.chmod(0o755)
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libga.so"))
    monkeypatch.setattr(build, "TENSORS", str(tmp_path / "_tensors.so"))
    monkeypatch.setattr(build, "HIPCC", str(linker))
    monkeypatch.setattr(build, "_compile", lambda src, verbose: src + ".o")

    def broken(verbose):
        raise FileNotFoundError("g++")

    monkeypatch.setattr(build, "_build_tensors", broken)
    with pytest.raises(FileNotFoundError):
        build.build()
    assert (tmp_path / "libga.so").read_text() == "linked\n"


@pytest.mark.parametrize("source", ["top", "distill", "balance"])
def test_launch_rules_fit_their_kernels(source, tmp_path):
    """Kernels load without masks where their launch rule says that every
    thread has its part: no row length gets a kernel that it does not fit, and
    a kernel that it does not fit is refused on the host."""
    from gradient_all_reduce_worker_amd import build

    obj = tmp_path / "rules.o"
    subprocess.run([build.HIPCC, "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-fPIC",
                    f"-D{source.upper()}", f'-DSOURCE="{os.path.join(build.CSRC, source + ".hip")}"', "-c",
                    os.path.join(ROOT, "tests", "launch_rules.cpp"), "-o", str(obj)], check=True)
    # the GPU code, which is not wanted (and not referred to, if the compiler sees through the stand-ins)
    undefined = subprocess.run(["nm", "-u", str(obj)], capture_output=True, text=True, check=True).stdout.split()
    (tmp_path / "image.c").write_text("".join(f"const char {s}[8] = {{0}};\n" for s in undefined if "fatbin" in s))
    subprocess.run(["gcc", "-c", str(tmp_path / "image.c"), "-o", str(tmp_path / "image.o")], check=True)
    subprocess.run(["g++", str(obj), str(tmp_path / "image.o"), "-o", str(tmp_path / "rules")], check=True)
    r = subprocess.run([str(tmp_path / "rules")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
