"""Host-side tests of the operators around the recurrence: argument refusals (every
one before any device call, so without a GPU), workspace sizes, and the fp64
references' gradients against central differences."""
import ctypes

import numpy as np
import pytest

import chunked_gated_delta_14_amd as gdr
import layer_ref as ref
from chunked_gated_delta_14_amd import layer

IN, OUT, OUT2 = 1 << 20, 1 << 21, 1 << 22
PTR = 4096  # never dereferenced: every call below is refused, or stops at the device check


def conv(**kw):
    f = dict(T=128, N=1, C=16, W=4, dtype=0, w_dtype=0, activation=1, n_chunks=2, x_stride=16, x=PTR, weight=PTR, bias=PTR, s0=PTR,
             chunk_table=PTR)
    f.update(kw)
    return layer._CConv(**f)


def gate(**kw):
    f = dict(T=128, H=2, D=128, dtype=0, kind=0, floor=-5.0, x_stride=256, x=PTR, a_log=PTR, bias=PTR)
    f.update(kw)
    return layer._CGate(**f)


def step(**kw):
    f = dict(T=4, N=4, H_qk=2, H_v=2, K=128, V=128, n_slots=4, input_flags=0, scale=0.1, q_stride=256, k_stride=256, v_stride=256,
             q=PTR, k=PTR, v=PTR, g=PTR, beta=PTR, cu_seqlens=None, slots=None, state=PTR)
    f.update(kw)
    return layer._CStep(**f)


def norm(**kw):
    f = dict(T=8, H=2, D=128, dtype=0, res_dtype=0, w_dtype=1, activation=1, placement=0, scale=1.0, eps=1e-6, x_stride=256,
             gate_stride=256, x=PTR, weight=PTR, gate=PTR, residual=None, s=None)
    f.update(kw)
    return layer._CNorm(**f)


def refused(rc, code, word):
    assert rc == code, (rc, gdr.lib().gdr_last_error().decode())
    assert word in gdr.lib().gdr_last_error().decode(), gdr.lib().gdr_last_error().decode()


BIG = 1 << 40


@pytest.mark.parametrize("kw,code,word", [
    (dict(T=-1), 1, "T and N"), (dict(C=0), 1, "C must"), (dict(C=1 << 25, x_stride=1 << 25), 2, "2^24"), (dict(W=1), 2, "W"),
    (dict(W=9), 2, "W"), (dict(dtype=2), 1, "dtype"), (dict(w_dtype=-1), 1, "dtype"), (dict(activation=2), 1, "activation"),
    (dict(x_stride=15), 1, "x_stride"), (dict(x=None), 1, "x and weight"), (dict(weight=None), 1, "x and weight"),
    (dict(x=PTR + 1), 1, "aligned"), (dict(bias=PTR + 1), 1, "aligned"), (dict(n_chunks=1), 1, "n_chunks"),
    (dict(n_chunks=4), 1, "n_chunks"), (dict(N=0), 1, "documents"), (dict(chunk_table=None), 1, "chunk_table"),
])
def test_conv_refusals(kw, code, word):
    L, p = gdr.lib(), conv(**kw)
    refused(L.gdr_conv_fwd(ctypes.byref(p), OUT, 1 << 26, None, None), code, word)
    refused(L.gdr_conv_bwd(ctypes.byref(p), PTR, 1 << 26, None, OUT, 1 << 26, PTR, None, None, PTR, BIG, None), code, word)


def test_conv_call_refusals():
    L, p = gdr.lib(), conv()
    r = ctypes.byref(p)
    refused(L.gdr_conv_fwd(None, PTR, 16, None, None), 1, "NULL")
    refused(L.gdr_conv_fwd(r, None, 16, None, None), 1, "y is NULL")
    refused(L.gdr_conv_fwd(r, PTR, 8, None, None), 1, "y_stride")
    refused(L.gdr_conv_fwd(r, PTR, 16, PTR + 1, None), 1, "aligned")
    need = gdr.conv_workspace_bytes(2, 16, 4, 0)
    assert need > 0 and need % 256 == 0
    refused(L.gdr_conv_bwd(r, PTR, 16, None, PTR, 16, None, None, None, PTR, need, None), 1, "dweight")
    refused(L.gdr_conv_bwd(r, None, 16, None, PTR, 16, PTR, None, None, PTR, need, None), 1, "dy and dx")
    refused(L.gdr_conv_bwd(r, PTR, 16, None, PTR, 15, PTR, None, None, PTR, need, None), 1, "stride")
    refused(L.gdr_conv_bwd(r, PTR, 16, None, OUT, 16, PTR, None, None, PTR, need - 1, None), 3, "too small")
    refused(L.gdr_conv_bwd(r, PTR, 16, None, OUT, 16, PTR, None, None, PTR + 16, need, None), 3, "aligned")
    refused(L.gdr_conv_bwd(r, PTR, 16, None, OUT, 16, PTR, None, None, None, need, None), 3, "NULL")
    q = conv(T=3, N=3)
    s = ctypes.byref(q)
    refused(L.gdr_conv_step(r, PTR, 16, PTR, PTR, 4, None), 1, "N must equal T")
    refused(L.gdr_conv_step(s, PTR, 16, PTR, None, 2, None), 1, "fewer slots")
    refused(L.gdr_conv_step(s, PTR, 16, PTR, PTR, -1, None), 1, "n_slots")
    refused(L.gdr_conv_step(s, PTR, 16, None, PTR, 3, None), 1, "state")
    refused(L.gdr_conv_step(s, PTR, 4, PTR, PTR, 3, None), 1, "y_stride")
    for bad in ((-1, 16, 4, 0), (2, 0, 4, 0), (2, 16, 4, 5), (2, 16, 9, 0)):
        with pytest.raises(gdr.GdrError):
            gdr.conv_workspace_bytes(*bad)


@pytest.mark.parametrize("kw,code,word", [
    (dict(T=-1), 1, "T must"), (dict(H=0), 1, "H must"), (dict(D=64), 2, "1 or 128"), (dict(H=70000, D=1), 2, "65536"),
    (dict(dtype=3), 1, "dtype"), (dict(kind=2), 1, "kind"), (dict(floor=0.0), 1, "floor"), (dict(floor=-8.5), 1, "floor"),
    (dict(floor=float("nan")), 1, "floor"), (dict(x_stride=255), 1, "x_stride"), (dict(x=None), 1, "x and a_log"),
    (dict(a_log=PTR + 2), 1, "aligned"),
])
def test_gate_refusals(kw, code, word):
    L, p = gdr.lib(), gate(**kw)
    refused(L.gdr_gate_fwd(ctypes.byref(p), PTR, None), code, word)
    refused(L.gdr_gate_bwd(ctypes.byref(p), PTR, PTR, 1 << 24, PTR, None, PTR, BIG, None), code, word)


def test_gate_call_refusals():
    L, p = gdr.lib(), gate()
    r, need = ctypes.byref(p), gdr.gate_workspace_bytes(128, 2, 128, 0)
    refused(L.gdr_gate_fwd(r, None, None), 1, "g is NULL")
    refused(L.gdr_gate_bwd(r, PTR, PTR, 256, None, None, PTR, need, None), 1, "da_log")
    refused(L.gdr_gate_bwd(r, PTR, None, 256, PTR, None, PTR, need, None), 1, "dg and dx")
    refused(L.gdr_gate_bwd(r, PTR, PTR, 200, PTR, None, PTR, need, None), 1, "dx_stride")
    refused(L.gdr_gate_bwd(r, PTR, OUT, 256, PTR, None, PTR, need - 256, None), 3, "too small")


@pytest.mark.parametrize("kw,code,word", [
    (dict(T=-1, N=-1), 1, ">= 0"), (dict(H_qk=0), 1, "head"), (dict(K=64), 2, "128"), (dict(N=3), 1, "N must equal T"),
    (dict(n_slots=3), 1, "fewer slots"), (dict(scale=float("nan")), 1, "scale"), (dict(input_flags=4), 1, "flag"),
    (dict(q_stride=255), 1, "stride"), (dict(v=None), 1, "non-NULL"), (dict(state=None), 1, "state is NULL"),
    (dict(state=PTR + 4), 1, "16-byte"), (dict(slots=PTR + 2), 1, "aligned"),
    (dict(H_qk=65537, H_v=65537, q_stride=1 << 24, k_stride=1 << 24, v_stride=1 << 24), 2, "too large"),
])
def test_step_refusals(kw, code, word):
    p = step(**kw)
    refused(gdr.lib().gdr_kda_step(ctypes.byref(p), PTR, None), code, word)
    refused(gdr.lib().gdr_gdn_step(ctypes.byref(p), PTR, None), code, word)


def test_step_head_groups():
    L = gdr.lib()
    refused(L.gdr_kda_step(ctypes.byref(step(H_v=4, v_stride=512)), PTR, None), 2, "KDA")
    refused(L.gdr_gdn_step(ctypes.byref(step(H_v=3, v_stride=512)), PTR, None), 2, "GDN")
    refused(L.gdr_kda_step(ctypes.byref(step()), None, None), 1, "non-NULL")


@pytest.mark.parametrize("kw,code,word", [
    (dict(T=-1), 1, "T must"), (dict(D=0), 1, "positive"), (dict(D=16385), 2, "16384"), (dict(dtype=2), 1, "dtype"),
    (dict(placement=3), 1, "placement"), (dict(activation=0), 1, "activation"), (dict(gate=None), 1, "activation"),
    (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"), (dict(scale=float("nan")), 1, "scale"),
    (dict(x=None), 1, "x is NULL"), (dict(x_stride=100), 1, "x_stride"), (dict(gate_stride=100), 1, "gate_stride"),
    (dict(placement=1, dtype=1, res_dtype=0, residual=PTR, s=PTR), 2, "bf16 residual"),
    (dict(placement=1, residual=PTR), 1, "s is NULL"), (dict(weight=PTR + 2), 1, "aligned"),
])
def test_norm_refusals(kw, code, word):
    L, p = gdr.lib(), norm(**kw)
    refused(L.gdr_norm_fwd(ctypes.byref(p), PTR, None), code, word)
    refused(L.gdr_norm_bwd(ctypes.byref(p), PTR, None, PTR, 256, PTR, 256, PTR if kw.get("placement") == 1 else None, PTR, PTR, BIG, None),
            code, word)


def test_norm_call_refusals():
    L, p = gdr.lib(), norm()
    r, need = ctypes.byref(p), gdr.norm_workspace_bytes(8, 2, 128)
    refused(L.gdr_norm_fwd(r, None, None), 1, "y is NULL")
    refused(L.gdr_norm_fwd(ctypes.byref(norm(placement=2)), PTR, None), 1, "residual is NULL")
    refused(L.gdr_norm_bwd(r, PTR, PTR, PTR, 256, PTR, 256, None, PTR, PTR, need, None), 1, "GDR_RES_BEFORE")
    refused(L.gdr_norm_bwd(r, PTR, None, PTR, 256, None, 256, None, PTR, PTR, need, None), 1, "dgate is NULL")
    refused(L.gdr_norm_bwd(r, PTR, None, None, 256, PTR, 256, None, PTR, PTR, need, None), 1, "dx is NULL")
    refused(L.gdr_norm_bwd(r, PTR, None, PTR, 256, PTR, 255, None, PTR, PTR, need, None), 1, "dgate_stride")
    refused(L.gdr_norm_bwd(r, PTR, None, OUT, 256, OUT2, 256, None, PTR, PTR, need - 256, None), 3, "too small")
    q = norm(gate=None, activation=0)
    refused(L.gdr_norm_bwd(ctypes.byref(q), PTR, None, PTR, 256, PTR, 256, None, PTR, PTR, need, None), 1, "dgate without")
    b = norm(placement=1, x=None, s=PTR)
    refused(L.gdr_norm_bwd(ctypes.byref(b), PTR, None, PTR, 256, PTR, 256, None, PTR, PTR, need, None), 1, "dres is NULL")


def test_conv_backward_of_empty_documents_needs_a_weight():
    """ds0 of documents without tokens launches a kernel, so a NULL weight is refused there too.  Without ds0, or without
    documents, nothing reads it and the call passes on to the check that follows, of a misaligned workspace."""
    L = gdr.lib()
    for N, ds0, code, word in ((3, OUT2, 1, "weight"), (3, None, 3, "aligned"), (0, OUT2, 3, "aligned")):
        p = conv(N=N, T=0, n_chunks=0, x=None, weight=None)
        refused(L.gdr_conv_bwd(ctypes.byref(p), None, 16, None, None, 16, OUT, None, ds0, PTR + 16, BIG, None), code, word)


def test_launch_limits():
    """A launch holds fewer than 2^32 threads and counts its rows, runs and documents with 32 bits: calls past that are
    refused by the checks.  The largest accepted sizes pass on to the check that follows, of an output off its alignment."""
    L = gdr.lib()

    def fwd(st, **kw):
        p = conv(x_stride=kw["C"], **kw)
        return L.gdr_conv_fwd(ctypes.byref(p), OUT + 1, kw["C"], OUT2 if st else None, None)

    # 2048 bf16 channels fill a block of 256 threads: 8 runs of each chunk (4 with W > 4), and a block for each final row
    for n, W, st, ok in ((2 ** 21 - 1, 4, False, True), (2 ** 21, 4, False, False), (2 ** 21 - 1, 4, True, False),
                         (2 ** 22 - 1, 5, False, True), (2 ** 22, 5, False, False)):
        rc = fwd(st, T=n, N=n, n_chunks=n, C=2048, W=W)
        refused(rc, *((1, "aligned") if ok else (2, "one launch")))
    # narrow rows: 256 sets to a block (C = 1), 85 (C = 3)
    most = 2 ** 28 - 32
    for n, C, ok in ((most, 1, True), (most + 31, 1, False), (2 ** 28 - 1, 3, False), (2 ** 24 * 85 // 8 - 86, 3, True)):
        rc = fwd(False, T=n, N=n, n_chunks=n, C=C)
        refused(rc, *((1, "aligned") if ok else (2, "one launch")))
    # the backward: a block of 256 threads for each half of ds0's rows beside the 16 workers' of 2 chunks in
    # runs of 8 tokens
    for N, ds0, ok in ((2 ** 23 - 17, True, True), (2 ** 23 - 16, True, False), (2 ** 23, False, True)):
        p = conv(N=N, C=2048, x_stride=2048)
        rc = L.gdr_conv_bwd(ctypes.byref(p), IN, 2048, None, OUT + 1, 2048, OUT2, None, OUT if ds0 else None, 1 << 24, BIG, None)
        refused(rc, *((1, "aligned") if ok else (2, "one launch")))
    # the parameter sums: (W + 1) C columns, 32 to a block of 1024 threads
    for W, ok in ((6, True), (7, False), (8, False)):
        p = conv(C=1 << 24, x_stride=1 << 24, W=W)
        rc = L.gdr_conv_bwd(ctypes.byref(p), IN, 1 << 24, None, OUT + 1, 1 << 24, OUT2, None, None, 1 << 24, BIG, None)
        refused(rc, *((1, "aligned") if ok else (2, "one launch")))
        if ok:
            assert gdr.conv_workspace_bytes(2, 1 << 24, W, 0) > 0
        else:
            with pytest.raises(gdr.GdrError):
                gdr.conv_workspace_bytes(2, 1 << 24, W, 0)
    for N, ok in ((2 ** 24 - 1, True), (2 ** 24, False)):
        p = conv(T=N, N=N, C=2048, x_stride=2048)
        rc = L.gdr_conv_step(ctypes.byref(p), OUT + 1, 2048, OUT2, PTR, 4, None)
        refused(rc, *((1, "aligned") if ok else (2, "one launch")))
    for N, ok in ((2 ** 20 - 1, True), (2 ** 20, False)):
        p = step(T=N, N=N, H_qk=16, H_v=16, q_stride=2048, k_stride=2048, v_stride=2048, slots=PTR + 2)
        refused(L.gdr_kda_step(ctypes.byref(p), OUT, None), *((1, "aligned") if ok else (2, "too large")))


def test_outputs_that_are_inputs_are_refused():
    """Each output given the address of one of the call's inputs."""
    L = gdr.lib()
    A, B, C, D, E = (IN + 4096 * i for i in range(5))
    c = ctypes.byref(conv(x=A, s0=B))
    for y, st in ((A, OUT), (B, OUT), (OUT, A), (OUT, B)):
        refused(L.gdr_conv_fwd(c, y, 16, st, None), 1, "is an input")
    ws = 1 << 24
    for dx, ds0 in ((A, OUT), (B, OUT), (C, OUT), (D, OUT), (OUT, A), (OUT, B), (OUT, C), (OUT, D)):
        refused(L.gdr_conv_bwd(c, C, 16, D, dx, 16, OUT2, None, ds0, ws, BIG, None), 1, "is an input")
    s = ctypes.byref(conv(T=3, N=3, x=A))
    for y, state in ((A, B), (B, B), (OUT, A)):
        refused(L.gdr_conv_step(s, y, 16, state, None, 3, None), 1, "is an input")
    g = ctypes.byref(gate(x=A, dtype=1))
    refused(L.gdr_gate_fwd(g, A, None), 1, "is an input")
    for dx in (A, B):
        refused(L.gdr_gate_bwd(g, B, dx, 256, OUT2, None, ws, BIG, None), 1, "is an input")
    t = ctypes.byref(step(q=A, k=B, v=C, state=D))
    for o in (A, B, C, D):
        refused(L.gdr_gdn_step(t, o, None), 1, "is an input")
    for y, q in ((A, norm(x=A, gate=B)), (B, norm(x=A, gate=B)), (C, norm(x=A, gate=B, placement=2, residual=C)),
                 (D, norm(x=A, gate=B, placement=1, residual=C, s=D)), (OUT, norm(x=A, gate=B, placement=1, residual=C, s=C))):
        refused(L.gdr_norm_fwd(ctypes.byref(q), y, None), 1, "is an input")
    b = ctypes.byref(norm(x=None, gate=B, placement=1, s=D))
    outs = [OUT, OUT2, OUT2 + 4096]
    for i in range(3):
        for bad in (B, C, D, E):
            dx, dz, dres = (bad if j == i else o for j, o in enumerate(outs))
            refused(L.gdr_norm_bwd(b, C, E, dx, 256, dz, 256, dres, None, None, 0, None), 1, "is an input")


def test_parameters_and_indices_are_not_outputs():
    """The same for every other pair: parameters, their gradients, tables, slots and the step's gates."""
    L, ws = gdr.lib(), 1 << 24
    A, B, C, D, E, F, G = (IN + 4096 * i for i in range(7))
    outs = [OUT + 4096 * i for i in range(4)]

    def each(n, ins):
        """The n outputs with one of them, in turn, one of the inputs."""
        for i in range(n):
            for bad in ins:
                yield [bad if j == i else o for j, o in enumerate(outs[:n])]

    c = ctypes.byref(conv(x=A, s0=B, weight=C, bias=D, chunk_table=E))
    for y, st in each(2, (A, B, C, D, E)):
        refused(L.gdr_conv_fwd(c, y, 16, st, None), 1, "is an input")
    for dx, dw, db, ds0 in each(4, (A, B, C, D, E, F, G)):
        refused(L.gdr_conv_bwd(c, F, 16, G, dx, 16, dw, db, ds0, ws, BIG, None), 1, "is an input")
    s = ctypes.byref(conv(T=3, N=3, x=A, weight=C, bias=D))
    for y, state in each(2, (A, C, D, E)):
        refused(L.gdr_conv_step(s, y, 16, state, E, 3, None), 1, "is an input")
    g = ctypes.byref(gate(x=A, a_log=B, bias=C, dtype=1))
    for out in (A, B, C):
        refused(L.gdr_gate_fwd(g, out, None), 1, "is an input")
    for dx, da, db in each(3, (A, B, C, D)):
        refused(L.gdr_gate_bwd(g, D, dx, 256, da, db, ws, BIG, None), 1, "is an input")
    for o, state in each(2, (A, B, C, D, E, F, G)):
        t = step(N=2, q=A, k=B, v=C, g=D, beta=E, cu_seqlens=F, slots=G, state=state)
        refused(L.gdr_kda_step(ctypes.byref(t), o, None), 1, "is an input")
        refused(L.gdr_gdn_step(ctypes.byref(t), o, None), 1, "is an input")
    for y, stream in each(2, (A, B, C, D)):
        n = norm(x=A, weight=B, gate=C, residual=D, s=stream, placement=1)
        refused(L.gdr_norm_fwd(ctypes.byref(n), y, None), 1, "is an input")
    n = ctypes.byref(norm(x=None, weight=B, gate=C, s=D, placement=1))
    for dx, dz, dres, dw in each(4, (B, C, D, E, F)):
        refused(L.gdr_norm_bwd(n, E, F, dx, 256, dz, 256, dres, dw, ws, BIG, None), 1, "is an input")


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    import torch

    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    for build in (lambda: gdr.ConvProblem(x, torch.zeros(16, 4), None), lambda: gdr.ConvStep(x, torch.zeros(16, 4), x),
                  lambda: gdr.GateProblem(x, torch.zeros(16)), lambda: gdr.NormProblem(x, None),
                  lambda: gdr.NormProblem(None, None),
                  lambda: gdr.StepProblem(gdr.GDR_KDA, x, x, x, x, x, x)):
        with pytest.raises(gdr.GdrError) as e:
            build()
        assert e.value.status == 1


def test_binding_refuses_sizes_past_32_bits():
    """A size that the C structs cannot hold is refused, not cut to its low 32 bits (2^32 + 8 rows are no 8 rows)."""
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode

    far = (1 << 32) + 8
    for call in (lambda: gdr.conv_workspace_bytes(far, 16, 4, 0), lambda: gdr.gate_workspace_bytes(far, 2, 128, 0),
                 lambda: gdr.norm_workspace_bytes(far, 1, 128), lambda: gdr.norm_workspace_bytes(8, far, 128)):
        with pytest.raises(gdr.GdrError, match="32 bits") as e:
            call()
        assert e.value.status == 1
    bf, i32 = torch.bfloat16, torch.int32
    with FakeTensorMode():  # shapes without memory

        def t(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device="cuda")

        class Plan:
            N, T, n_chunks, table = 1, far, far // 64, None

        one = [t(1, 1, 128, dtype=bf)] * 3
        for build in (lambda: gdr.ConvProblem(t(far, 1), t(1, 4), Plan),
                      lambda: gdr.ConvStep(t(far, 1), t(1, 4), t(4, 3, 1), t(far, dtype=i32)),
                      lambda: gdr.ConvStep(t(2, 1), t(1, 4), t(far, 3, 1), t(2, dtype=i32)),
                      lambda: gdr.GateProblem(t(far, 1), t(1)), lambda: gdr.NormProblem(t(far, 1), None),
                      lambda: gdr.NormProblem(t(2, far, 1), None),
                      lambda: gdr.StepProblem(gdr.GDR_GDN, *[t(far, 1, 128, dtype=bf)] * 3, t(far, 1), t(far, 1), t(4, 1, 128, 128)),
                      lambda: gdr.StepProblem(gdr.GDR_GDN, *one, t(1, 1), t(1, 1), t(far, 1, 128, 128), None, t(1, dtype=i32)),
                      lambda: gdr.StepProblem(gdr.GDR_GDN, *one, t(1, 1), t(1, 1), t(4, 1, 128, 128), t(far + 1, dtype=i32))):
            with pytest.raises(gdr.GdrError, match="32 bits") as e:
                build()
            assert e.value.status == 1


def test_binding_row_checks():
    """The row checks work on any device's tensors: strides, overlaps and types."""
    import torch

    dev = torch.device("cpu")
    wide = torch.zeros(6, 40)
    assert layer._rows(wide[:, :16], "x", (6, 16), torch.float32, dev) == 40
    assert layer._rows(wide[:1, :16], "x", None, None, dev) == 16
    assert layer._rows(wide[:, :32].unflatten(1, (2, 16)), "x", None, None, dev) == 40
    for t in (wide.t(), wide[:, ::2], wide[:, :32].unflatten(1, (2, 16)).transpose(1, 2), torch.zeros(16).expand(6, 16)):
        with pytest.raises(gdr.GdrError):
            layer._rows(t, "x", None, None, dev)
    with pytest.raises(gdr.GdrError):
        layer._rows(wide, "x", (6, 41), None, dev)
    with pytest.raises(gdr.GdrError):
        layer._need(wide, "x", None, torch.bfloat16, dev)


# ---- the references' gradients against central differences ----


def differences(f, args, names, h=1e-6):
    """d f / d args[name] by central differences, for a scalar f."""
    out = {}
    for n in names:
        a = args[n]
        g = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = f()
            a[i] = keep - h
            g[i] = (up - f()) / (2 * h)
            a[i] = keep
        out[n] = g
    return out


def agree(got, want):
    # central differences of O(1) sums: truncation h^2 and rounding 1e-16 / h, both well below 1e-7
    assert np.max(np.abs(got - want)) <= 1e-7 * (1 + np.max(np.abs(want)))


@pytest.mark.parametrize("silu", [True, False])
def test_conv_reference_gradient(silu):
    r, docs, C, W = np.random.default_rng(3), (5, 0, 1, 2), 3, 4
    a = dict(x=r.standard_normal((8, C)), w=r.standard_normal((C, W)), b=r.standard_normal(C), s0=r.standard_normal((4, W - 1, C)))
    dy, dst = r.standard_normal((8, C)), r.standard_normal((4, W - 1, C))

    def loss():
        f = ref.conv(a["x"], a["w"], a["b"], a["s0"], docs, silu)
        return (f["y"] * dy).sum() + (f["st"] * dst).sum()

    d = ref.conv_grad(ref.conv(a["x"], a["w"], a["b"], a["s0"], docs, silu), a["x"], a["w"], docs, dy, dst, silu)
    n = differences(loss, a, a)
    for key, name in (("x", "dx"), ("w", "dw"), ("b", "db"), ("s0", "ds0")):
        agree(d[name], n[key])


@pytest.mark.parametrize("kind", ["softplus", "sigmoid"])
def test_gate_reference_gradient(kind):
    r = np.random.default_rng(4)
    a = dict(x=r.standard_normal((5, 2, 3)), a=r.standard_normal(2), b=r.standard_normal((2, 3)))
    dg = r.standard_normal((5, 2, 3))
    n = differences(lambda: (ref.gate(a["x"], a["a"], a["b"], kind, -5.0)[0] * dg).sum(), a, a)
    d = ref.gate_grad(a["x"], a["a"], a["b"], kind, -5.0, dg)
    for key, name in (("x", "dx"), ("a", "da"), ("b", "db")):
        agree(d[name], n[key])


@pytest.mark.parametrize("place,act", [("none", "none"), ("none", "silu"), ("before", "sigmoid"), ("after", "silu")])
def test_norm_reference_gradient(place, act):
    r, shape, alpha = np.random.default_rng(5), (3, 2, 5), 0.7
    a = dict(x=r.standard_normal(shape), w=r.standard_normal(5), z=r.standard_normal(shape), res=r.standard_normal(shape))
    dy, ds = r.standard_normal(shape), r.standard_normal(shape)
    z = a["z"] if act != "none" else None

    def loss():
        f = ref.norm(a["x"], a["w"], z, a["res"], place, act, alpha, 1e-3)
        return (f["y"] * dy).sum() + ((f["s"] * ds).sum() if place == "before" else 0.0)

    u = ref.norm(a["x"], a["w"], z, a["res"], place, act, alpha, 1e-3)["s"] if place == "before" else a["x"]
    d = ref.norm_grad(u, a["w"], z, dy, ds if place == "before" else None, place, act, alpha, 1e-3)
    n = differences(loss, a, a)
    agree(d["dx"], n["x"])
    agree(d["dw"], n["w"])
    if z is not None:
        agree(d["dz"], n["z"])
    if place == "before":
        agree(d["dres"], n["res"])
    if place == "after":
        agree(dy, n["res"])


def test_step_reference_equals_the_oracle():
    """Token by token from the same state: the step's reference and the recurrence's oracle."""
    import oracle

    r, docs = np.random.default_rng(6), (3, 1)
    T, H = 4, 2
    q, k = (t / np.linalg.norm(t, axis=-1, keepdims=True) for t in r.standard_normal((2, T, 1, 128)))
    v, g, beta = r.standard_normal((T, H, 128)), -r.random((T, H)), r.random((T, H))
    h0 = 0.1 * r.standard_normal((2, H, 128, 128))
    o, ht = oracle.forward(q, k, v, g, beta, np.array([0, 3, 4], np.int32), h0)
    ro, _, rs, _ = ref.step(q, k, v, g, beta, h0.copy(), docs, [0, 1], 128 ** -0.5, False, False)
    assert np.allclose(ro, o, rtol=0, atol=1e-12) and np.allclose(rs, ht, rtol=0, atol=1e-12)
