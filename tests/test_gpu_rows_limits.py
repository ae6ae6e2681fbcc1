"""A layer's row operators beside early starts of the kernels around them, and at the ends of what they take."""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_kv_pred_gb300 as bs
from _parity import ensure_built
from test_gpu_rows import D, bf16, i32, same, word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


# ---------------------------------------------------------------------------
# kernels that start early
# ---------------------------------------------------------------------------
LISTS = ("topk", "res", "cpu", "delta")


def selection_args(q, digest, seq, bits, B, Hq, Hkv, P, cap, k, out, ws, launch, stream):
    lists = [out[n + s].data_ptr() for n in LISTS for s in ("", "_count")]
    return (bs.MINMAX, q.data_ptr(), digest.data_ptr(), seq.data_ptr(), bits.data_ptr(), None, None, B, Hq, Hkv, D, P, cap, k,
            None, *lists, ws.data_ptr(), ws.numel(), None, launch, stream.cuda_stream)


@pytest.mark.parametrize("by", ["pdl", "event"])
def test_a_selection_that_starts_early_after_a_turned_prediction_finds_the_digests_before_it(by):
    """Digests, the rotated prediction as it is always launched, and a selection that streams digests before it waits
    for the prediction: those of the digest kernel, by either way to start early."""
    rng = np.random.default_rng(1)
    B, H, P, cap, k = 8, 8, 32, 512, 16
    rope = bs.rope(1e6, 128)
    K = torch.from_numpy(rng.standard_normal((B * H * cap, P, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    table = torch.arange(B * H * cap, dtype=torch.int32, device="cuda").view(B, H, cap)
    seq = i32([cap * P - 40 * b for b in range(B)])
    X, W, pos = bf16(rng, B, 512), bf16(rng, H * D, 512), seq - 1
    bits = torch.full((B, H, cap // 32), 0x55555555, dtype=torch.int32, device="cuda")
    digest = torch.zeros((B, H, cap, 2, D), dtype=torch.bfloat16, device="cuda")
    ws, Q = bs.score_topk_workspace(B, H, cap), torch.empty((B, H * D), dtype=torch.bfloat16, device="cuda")
    bs.build_digest("minmax", K, table, seq, B, H, P, digest)
    bs.predict_q_rotated(X, W, pos, rope, Q=Q)
    torch.cuda.synchronize()
    want = bs.score_topk("minmax", Q.view(B, H, D), digest, seq, bits, B, H, H, P, cap, k, ws)
    got = {n: torch.empty_like(t) for n, t in want.items()}
    args, L, st, other = bs.RopeArgs(rope.turns.data_ptr(), 128, 0, 1.0), bs.lib(), torch.cuda.Stream(), torch.cuda.Stream()
    event = torch.cuda.Event()
    event.record(st)
    first = None if by == "pdl" else bs._launch(0, early_event=event)
    second = bs._launch(0, pdl=True) if by == "pdl" else None
    for _ in range(20):
        digest.zero_(), Q.zero_()
        for t in got.values():
            t.fill_(-9)
        torch.cuda.synchronize()
        bs.build_digest("minmax", K, table, seq, B, H, P, digest, stream=st)
        assert L.scout_predict_q_rotated(X.data_ptr(), W.data_ptr(), Q.data_ptr(), B, H * D, 512, pos.data_ptr(), ctypes.byref(args),
                                         None, 1e-6, None, first, st.cuda_stream) == 0
        on = st
        if by == "event":
            on = other
            other.wait_event(event)
        assert L.scout_score_topk(*selection_args(Q, digest, seq, bits, B, H, H, P, cap, k, got, ws, second, on)) == 0
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]), n


def test_a_selection_over_empty_sequences_that_starts_early_writes_after_its_wait():
    """Its lists lie where the kernel before it writes: they are there last, whichever started first."""
    B, H, P, cap, k = 4, 2, 32, 64, 8
    rng = np.random.default_rng(2)
    M, N, K = 256, 128, 32768  # one CTA that streams 25 MB
    X, W = (torch.ones((n, K), dtype=torch.bfloat16, device="cuda") for n in (M, N))
    digest = torch.zeros((B, H, cap, 2, D), dtype=torch.bfloat16, device="cuda")
    q, bits = bf16(rng, B, H, D), torch.zeros((B, H, cap // 32), dtype=torch.int32, device="cuda")
    ws, L, st = bs.score_topk_workspace(B, H, cap), bs.lib(), torch.cuda.Stream()
    Q = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    words = Q.view(torch.int32).flatten()
    shapes = [(n + s, (B, H, k) if s == "" else (B, H)) for n in LISTS for s in ("", "_count")]
    out, at = {}, 0
    for n, shape in shapes:
        out[n] = words[at:at + int(np.prod(shape))].view(shape)
        at += int(np.prod(shape))
    for lens in ([0] * B, [0, -5, 0, -1]):
        seq = i32(lens)
        for _ in range(10):
            words.fill_(-9)
            torch.cuda.synchronize()
            assert L.scout_predict_q(X.data_ptr(), W.data_ptr(), Q.data_ptr(), M, N, K, None, bs._launch(1), st.cuda_stream) == 0
            assert L.scout_score_topk(*selection_args(q, digest, seq, bits, B, H, H, P, cap, k, out, ws, bs._launch(0, pdl=True), st)) == 0
            torch.cuda.synchronize()
            for n, shape in shapes:
                assert torch.all(out[n] == (0 if n.endswith("_count") else -1)), n
            assert torch.all(Q.flatten()[2 * at:] == float(K))


def test_a_captured_selection_that_starts_early_after_a_turned_prediction_and_a_joined_stream():
    """One graph: two streams joined before a row kernel, copies and fills between row kernels, digests, the rotated
    prediction, a selection that starts early.  Replayed over inputs that change."""
    rng = np.random.default_rng(3)
    B, H, P, cap, k, N = 8, 8, 32, 256, 16, 512
    rope = bs.rope(1e6, 128)
    K = torch.zeros((B * H * cap, P, D), dtype=torch.bfloat16, device="cuda")
    table = torch.arange(B * H * cap, dtype=torch.int32, device="cuda").view(B, H, cap)
    seq = i32([cap * P - 40 * b for b in range(B)])
    Y, S, W, w = bf16(rng, B, N), bf16(rng, B, N), bf16(rng, H * D, N), bf16(rng, N)
    pos, heads = torch.zeros_like(seq), bf16(rng, B, H, D)
    bits = torch.full((B, H, cap // 32), 0x55555555, dtype=torch.int32, device="cuda")
    digest = torch.zeros((B, H, cap, 2, D), dtype=torch.bfloat16, device="cuda")
    ws, Q = bs.score_topk_workspace(B, H, cap), torch.empty((B, H * D), dtype=torch.bfloat16, device="cuda")
    S2, X, R, R2 = torch.empty_like(S), torch.empty_like(Y), torch.empty_like(heads), torch.empty_like(heads)
    shape = {n + s: (B, H, k) if s == "" else (B, H) for n in LISTS for s in ("", "_count")}
    got = {n: torch.empty(s, dtype=torch.int32, device="cuda") for n, s in shape.items()}
    args, L = bs.RopeArgs(rope.turns.data_ptr(), 128, 0, 1.0), bs.lib()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    launch = bs._launch(0, pdl=True)

    def run(second):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            bs.add_norm("rms", Y, S, w, H_out=S2, X=X)
        with torch.cuda.stream(main):
            pos.copy_(seq).sub_(1)
            bs.rotate(heads, pos, rope, out=R)
            R2.copy_(R)
            bs.rotate(R2, pos, rope, out=R2)
            main.wait_stream(side)
            digest.fill_(0)
            bs.build_digest("minmax", K, table, seq, B, H, P, digest)
        assert L.scout_predict_q_rotated(X.data_ptr(), W.data_ptr(), Q.data_ptr(), B, H * D, N, pos.data_ptr(), ctypes.byref(args),
                                         None, 1e-6, None, None, main.cuda_stream) == 0
        assert L.scout_score_topk(*selection_args(Q, digest, seq, bits, B, H, H, P, cap, k, got, ws, second, main)) == 0

    run(None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        run(launch)
    for i in range(5):
        K.copy_(torch.from_numpy(rng.standard_normal(K.shape).astype(np.float32)))
        Y.copy_(bf16(rng, B, N)), heads.copy_(bf16(rng, B, H, D)), seq.sub_(17 * i)
        torch.cuda.synchronize()
        run(None)
        torch.cuda.synchronize()
        want = {n: t.clone() for n, t in got.items()} | {"Q": Q.clone(), "X": X.clone(), "R": R.clone(), "R2": R2.clone()}
        for t in (*got.values(), Q, X, R, R2):
            t.fill_(-9)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n, t in {**got, "Q": Q, "X": X, "R": R, "R2": R2}.items():
            assert same(t, want[n]), n
