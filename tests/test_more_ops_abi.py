"""C entries of the embedding, the gated recurrence and the losses without a GPU: sizes, and refusals, which come before any
CUDA call."""
import ctypes
import os
import shutil
import subprocess

import pytest

from fsdp2_gradient_packing_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(4096)       # a pointer that no refused call follows
ODD = ctypes.c_void_p(4098)
BIG = 1 << 40


@pytest.fixture(scope="module")
def fp():
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up pointers: only where no kernel could run on them")
    _build.build()
    from fsdp2_gradient_packing_gb300 import fsdp_pack
    return fsdp_pack


def refused(fp, status, want, word):
    assert status == want, fp.fsdp_last_error()
    assert word in fp.fsdp_last_error()


def embedding(fp, **k):
    d = dict(rows=10, vocab=50, cols=64, ld_weight=64, ld_out=64, token_dtype=1, weight_dtype=1, out_dtype=1, accumulate=0, scale=1.0)
    d.update(k)
    return ctypes.byref(fp.fsdp_embedding_desc_t(**d))


def test_embedding_refusals(fp):
    lib = fp._lib
    E, N = fp.FSDP_EINVAL, fp.FSDP_EUNSUPPORTED

    def forward(d, t=P, w=P, o=P):
        return lib.fsdp_embedding_forward(d, t, w, o, None)

    def backward(d, t=P, o=P, w=P, ws=P, n=BIG):
        return lib.fsdp_embedding_backward(d, t, o, w, ws, n, None)

    for call in (forward, backward):
        refused(fp, call(None), E, "desc")
        refused(fp, call(embedding(fp, rows=-1)), E, "rows")
        refused(fp, call(embedding(fp, vocab=0)), E, "vocab")
        refused(fp, call(embedding(fp, cols=0)), E, "cols")
        refused(fp, call(embedding(fp, rows=1 << 31)), N, "2^31")
        refused(fp, call(embedding(fp, vocab=(1 << 31) - 1)), N, "2^31")
        refused(fp, call(embedding(fp, vocab=1 << 30, cols=1 << 40)), N, "too large")
        refused(fp, call(embedding(fp, token_dtype=2)), E, "token_dtype")
        refused(fp, call(embedding(fp, weight_dtype=2)), E, "weight_dtype")
        refused(fp, call(embedding(fp, out_dtype=-1)), E, "out_dtype")
        refused(fp, call(embedding(fp, accumulate=2)), E, "accumulate")
        refused(fp, call(embedding(fp, scale=float("inf"))), E, "scale")
        refused(fp, call(embedding(fp, ld_weight=63)), E, "row distance")
        refused(fp, call(embedding(fp, ld_out=63)), E, "row distance")
        refused(fp, call(embedding(fp), t=None), E, "tokens is NULL")
        refused(fp, call(embedding(fp), t=ctypes.c_void_p(4100)), E, "tokens is not 8-byte")
        refused(fp, call(embedding(fp), w=None), E, "weight is NULL")
        refused(fp, call(embedding(fp, out_dtype=0), o=ODD), E, "4-byte aligned")
    assert forward(embedding(fp, rows=0), t=None, o=None) == fp.FSDP_OK
    refused(fp, backward(embedding(fp), n=0), E, "workspace_bytes")
    refused(fp, backward(embedding(fp), ws=None), E, "workspace is NULL")
    refused(fp, backward(embedding(fp), ws=ctypes.c_void_p(4104)), E, "16-byte")


def test_embedding_workspace(fp):
    assert fp.fsdp_embedding_workspace(0, 50, 64) == 0
    assert fp.fsdp_embedding_workspace(1000, 50, 64) >= 1000 * 8
    refused(fp, fp._lib.fsdp_embedding_workspace(embedding(fp), None), fp.FSDP_EINVAL, "bytes")


def scan(fp, **k):
    d = dict(rows=12, cols=64, seqs=3, seq_len=4, ld_x=64, ld_gate=64, ld_h=64, ld_dx=64, ld_dgate=64, packed=0, offset_dtype=0, x_dtype=1,
             h_dtype=1, dx_dtype=1, param_dtype=0, grad_dtype=0)
    d.update(k)
    return ctypes.byref(fp.fsdp_scan_desc_t(**d))


def test_scan_refusals(fp):
    lib = fp._lib
    E, N = fp.FSDP_EINVAL, fp.FSDP_EUNSUPPORTED

    def forward(d, x=P, g=P, b=P, i=P, o=None, h=P, f=P, s=P, ws=P, n=BIG):
        return lib.fsdp_gated_scan_forward(d, x, g, b, i, o, h, f, s, ws, n, None)

    def backward(d, h=P, x=P, g=P, b=P, i=P, o=None, s=P, df=P, dx=P, dg=P, db=P, di=ctypes.c_void_p(1 << 20), ws=P, n=BIG):
        return lib.fsdp_gated_scan_backward(d, h, x, g, b, i, o, s, df, dx, dg, db, di, ws, n, None)

    for call in (forward, backward):
        refused(fp, call(None), E, "desc")
        refused(fp, call(scan(fp, rows=-1)), E, "rows")
        refused(fp, call(scan(fp, cols=0)), E, "cols")
        refused(fp, call(scan(fp, seqs=-1)), E, "seqs")
        refused(fp, call(scan(fp, rows=13)), E, "seqs * seq_len")
        refused(fp, call(scan(fp, seqs=0)), E, "seqs * seq_len")
        refused(fp, call(scan(fp, seq_len=-4)), E, "seq_len")
        refused(fp, call(scan(fp, seqs=1 << 20, seq_len=1 << 50)), E, "seqs * seq_len")
        refused(fp, call(scan(fp, rows=1 << 31, seqs=1, seq_len=1 << 31)), N, "2^31")
        refused(fp, call(scan(fp, cols=1 << 60)), N, "too large")
        refused(fp, call(scan(fp, packed=2)), E, "packed")
        refused(fp, call(scan(fp, packed=1, offset_dtype=2), o=P), E, "offset_dtype")
        refused(fp, call(scan(fp, packed=1)), E, "offsets is NULL")
        refused(fp, call(scan(fp, packed=1, offset_dtype=1), o=ctypes.c_void_p(4100)), E, "offsets")
        refused(fp, call(scan(fp), o=P), E, "packed is 0")
        refused(fp, call(scan(fp, x_dtype=2)), E, "x_dtype")
        refused(fp, call(scan(fp, h_dtype=2)), E, "h_dtype")
        refused(fp, call(scan(fp, dx_dtype=3)), E, "dx_dtype")
        refused(fp, call(scan(fp, param_dtype=3)), E, "param_dtype")
        refused(fp, call(scan(fp, grad_dtype=3)), E, "grad_dtype")
        refused(fp, call(scan(fp, ld_gate=63)), E, "gate")
        refused(fp, call(scan(fp, ld_h=63)), E, "row distance")
        refused(fp, call(scan(fp), x=None), E, "x is NULL")
        refused(fp, call(scan(fp), h=None), E, "h is NULL")
        refused(fp, call(scan(fp), b=ODD), E, "bias")
        refused(fp, call(scan(fp), i=ODD), E, "initial")
        refused(fp, call(scan(fp), s=ODD), E, "states")
    refused(fp, forward(scan(fp), f=ODD), E, "final")
    refused(fp, backward(scan(fp), s=None), E, "states is NULL")
    refused(fp, backward(scan(fp), dx=None), E, "dx is NULL")
    refused(fp, backward(scan(fp), dg=None), E, "dgate is NULL")
    refused(fp, backward(scan(fp), db=ODD), E, "dbias")
    refused(fp, backward(scan(fp), df=ODD), E, "dfinal")
    refused(fp, backward(scan(fp), di=ODD), E, "dinitial")
    refused(fp, backward(scan(fp), di=P), E, "dinitial is dfinal")
    refused(fp, backward(scan(fp), n=0), E, "workspace_bytes")
    refused(fp, backward(scan(fp), ws=None), E, "workspace is NULL")
    assert forward(scan(fp, rows=0, seqs=0), x=None, g=None, h=None) == fp.FSDP_OK
    out = ctypes.c_int64()
    refused(fp, lib.fsdp_gated_scan_states(-1, 4, ctypes.byref(out)), E, "rows")
    refused(fp, lib.fsdp_gated_scan_states(4, 4, None), E, "n is NULL")
    assert fp.fsdp_gated_scan_states(0, 4) == 0 and fp.fsdp_gated_scan_states(1, 4) == 1 and fp.fsdp_gated_scan_states(1000, 4) >= 1


def distill(fp, **k):
    d = dict(rows=4, vocab=500, ld_logits=500, ld_dlogits=500, top=8, ld_tokens=8, ld_teacher=8, logits_dtype=1, dlogits_dtype=1,
             teacher_dtype=1, token_dtype=1, temperature=1.0)
    d.update(k)
    return ctypes.byref(fp.fsdp_distill_desc_t(**d))


def policy(fp, **k):
    d = dict(rows=4, vocab=500, ld_logits=500, ld_dlogits=500, logits_dtype=1, dlogits_dtype=1, token_dtype=1, temperature=1.0, clip_low=0.2,
             clip_high=0.2, kl=0.0)
    d.update(k)
    return ctypes.byref(fp.fsdp_policy_desc_t(**d))


def test_loss_refusals(fp):
    lib = fp._lib
    E, N = fp.FSDP_EINVAL, fp.FSDP_EUNSUPPORTED
    Q = ctypes.c_void_p(1 << 20)

    def dis_f(d, z=P, i=P, t=P, w=P, lo=P, e=P, g=Q):
        return lib.fsdp_distill_loss_forward(d, z, i, t, w, lo, e, g, None)

    def dis_b(d, z=P, i=P, t=P, w=P, e=P, u=P, g=Q):
        return lib.fsdp_distill_loss_backward(d, z, i, t, w, e, u, g, None)

    def pol_f(d, z=P, i=P, o=P, r=P, a=P, w=P, lo=P, lp=P, e=P, g=Q):
        return lib.fsdp_policy_loss_forward(d, z, i, o, r, a, w, lo, lp, e, g, None)

    def pol_b(d, z=P, i=P, o=P, r=P, a=P, w=P, lp=P, e=P, u=P, g=Q):
        return lib.fsdp_policy_loss_backward(d, z, i, o, r, a, w, lp, e, u, g, None)

    for call, desc in ((dis_f, distill), (dis_b, distill), (pol_f, policy), (pol_b, policy)):
        refused(fp, call(None), E, "desc")
        refused(fp, call(desc(fp, rows=-1)), E, "rows")
        refused(fp, call(desc(fp, vocab=0)), E, "vocab")
        refused(fp, call(desc(fp, vocab=1 << 31)), N, "2^31")
        refused(fp, call(desc(fp, vocab=(1 << 31) - 63)), N, "2^31")
        refused(fp, call(desc(fp, rows=1 << 55)), N, "too large")
        refused(fp, call(desc(fp, logits_dtype=2)), E, "logits_dtype")
        refused(fp, call(desc(fp, dlogits_dtype=2)), E, "dlogits_dtype")
        refused(fp, call(desc(fp, token_dtype=2)), E, "token_dtype")
        for t in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
            refused(fp, call(desc(fp, temperature=t)), E, "temperature")
        refused(fp, call(desc(fp, ld_logits=499)), E, "logits")
        refused(fp, call(desc(fp, ld_dlogits=499)), E, "dlogits")
        refused(fp, call(desc(fp), z=None), E, "logits is NULL")
        refused(fp, call(desc(fp, logits_dtype=0), z=ODD), E, "4-byte")
        refused(fp, call(desc(fp), i=None), E, "tokens is NULL")
        refused(fp, call(desc(fp), w=ODD), E, "weight")
        refused(fp, call(desc(fp), e=None), E, "lse is NULL")
        refused(fp, call(desc(fp, dlogits_dtype=0), g=P), E, "dlogits is logits")
        refused(fp, call(desc(fp, ld_dlogits=504), g=P), E, "dlogits is logits")
    for call in (dis_b, pol_b):
        refused(fp, call(distill(fp) if call is dis_b else policy(fp), g=None), E, "dlogits is NULL")
        refused(fp, call(distill(fp) if call is dis_b else policy(fp), u=ODD), E, "dloss")
    for call in (dis_f, dis_b):
        refused(fp, call(distill(fp, top=-1)), E, "top")
        refused(fp, call(distill(fp, top=1025, ld_tokens=1025, ld_teacher=1025)), N, "FSDP_DISTILL_MAX_TOP")
        refused(fp, call(distill(fp, teacher_dtype=2)), E, "teacher_dtype")
        refused(fp, call(distill(fp, ld_tokens=7)), E, "teacher_tokens")
        refused(fp, call(distill(fp, ld_teacher=7)), E, "teacher_logits")
        refused(fp, call(distill(fp), t=None), E, "teacher_logits is NULL")
    refused(fp, dis_f(distill(fp), lo=None), E, "loss is NULL")
    refused(fp, pol_f(policy(fp), lo=None), E, "loss is NULL")
    for call in (pol_f, pol_b):
        refused(fp, call(policy(fp), lp=None), E, "logp is NULL")
        refused(fp, call(policy(fp), a=None), E, "advantage is NULL")
        refused(fp, call(policy(fp), o=ODD), E, "old_logp")
        refused(fp, call(policy(fp), r=ODD), E, "ref_logp")
        refused(fp, call(policy(fp, clip_low=-1.0)), E, "clip_low")
        refused(fp, call(policy(fp, clip_high=float("nan"))), E, "clip_low or clip_high")
        refused(fp, call(policy(fp, kl=float("inf"))), E, "kl")
    assert dis_f(distill(fp, rows=0), z=None, i=None, t=None, lo=None, e=None, g=None) == fp.FSDP_OK
    assert pol_f(policy(fp, rows=0), z=None, i=None, a=None, lo=None, lp=None, e=None, g=None) == fp.FSDP_OK


def test_header_in_strict_c(tmp_path):
    if not shutil.which("gcc"):
        pytest.skip("gcc is not installed")
    src = tmp_path / "ops.c"
    src.write_text('#include "fsdp_ops.h"\nint main(void) { return sizeof(fsdp_embedding_desc_t) == 64 && sizeof(fsdp_scan_desc_t) == 104 && '
                   'sizeof(fsdp_distill_desc_t) == 80 && sizeof(fsdp_policy_desc_t) == 64 ? 0 : 1; }\n')
    exe = tmp_path / "ops"
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
