"""States whose memory is held in 8 bits, reordering of a state's rows, and beam search over a
state, against the oracle.

Half steps: e4m3 2^-4 of a normal value, 2^-10 of a scale below 2^-6 scales.  The fp32 path's
tolerance against the fp64 oracle is 1e-4, the bf16 path's 3e-2 (rlt_testlib).
"""
import math

import numpy as np
import pytest

import rlt_inputs as ri
from oracle.rlt_oracle import RLTOracle
from tests.rlt_testlib import oracle_mode, tol_for

pytestmark = pytest.mark.gpu

BASE = ri.RLTConfig("small", vocab=40, d=128, heads=2, n_enc=2, n_dec=2, ffn=256, window=8, groups=2,
                    chunk=1, variant=1, tied=0, dtype=ri.DT_F32)
# the weights of the other tests give nearly uniform logits; wider ones spread them
STD = 0.2


@pytest.fixture(scope="module")
def sd():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tests.conftest import build_library
    build_library()
    import stateful_decoding_b200 as sd
    return sd


def _model(sd, cfg, std=0.02):
    w = ri.generate_weights(cfg, seed=7, std=std)
    blob = ri.write_blob(cfg, w, seed=7)
    return sd.Model(blob), RLTOracle(cfg, ri.read_blob(blob)[1], oracle_mode(cfg))


def _tokens(cfg, rows, n, seed=1):
    return np.random.default_rng(seed).integers(0, cfg.vocab, (rows, n)).astype(np.int32)


def _memory(sd, st, cfg):
    """[G][B][2][h][positions][dh] of an 8-bit memory, in fp64, and its scales [G][B][P][2][h]."""
    import torch
    G, B, h, dh = cfg.groups, st.batch, cfg.heads, cfg.d // cfg.heads
    P = -(-st.max_len // 64)
    sc = st.read(sd.PART_MEM_SCALES).view(np.float32).astype(np.float64).reshape(G, B, P, 2, h)
    x = torch.from_numpy(st.read(sd.PART_MEM)).view(torch.float8_e4m3fn).double().numpy()
    x = x.reshape(G, B, P, 2, h, 64, dh) * sc[..., None, None]
    return x.transpose(0, 1, 3, 4, 2, 5, 6).reshape(G, B, 2, h, P * 64, dh), sc


@pytest.mark.parametrize("kw,pieces", [
    (dict(), [70]), (dict(), [1, 62, 1, 1, 20]), (dict(d=128, heads=1, groups=1), [130]),
    (dict(dtype=ri.DT_BF16), [3, 64]), (dict(dtype=ri.DT_BF16, d=256), [1, 1, 1])])
def test_memory_holds_the_oracles_keys_and_values(sd, kw, pieces):
    cfg = BASE.replace(**kw)
    model, oracle = _model(sd, cfg)
    st = sd.State(model, 3, 200, mem8=True)
    tok = _tokens(cfg, 3, sum(pieces))
    at = 0
    for n in pieces:
        st.encode(np.ascontiguousarray(tok[:, at:at + n]))
        at += n
    st.check()
    got, scales = _memory(sd, st, cfg)
    tol = tol_for(cfg)
    for b in range(3):
        row = oracle.new_state()
        oracle.encode(row, tok[b])
        for g in range(cfg.groups):
            for w, want in enumerate((row.mem_k[g], row.mem_v[g])):
                want = want.transpose(1, 0, 2)                   # [h][positions][dh]
                s = scales[g, b, :, w][np.arange(at) // 64].T[..., None]
                # rounded once, and again below the subnormal border when a page's scale grew
                err = np.abs(got[g, b, w][:, :at] - want)
                assert (err <= np.abs(want) * 2.0 ** -4 + s * 2.0 ** -9 + tol).all(), (b, g, w, err.max())
                for p in range(-(-at // 64)):
                    top = np.abs(want[:, 64 * p:64 * p + 64]).max((1, 2))
                    sp = scales[g, b, p, w]
                    assert (np.log2(sp) == np.round(np.log2(sp))).all()
                    assert (top <= 448 * sp + tol).all() and (top + tol > 224 * sp).all()


@pytest.mark.parametrize("kw,T", [
    (dict(), 5), (dict(d=128, heads=1, groups=1), 70), (dict(variant=2, chunk=6), 20),
    (dict(variant=0), 40), (dict(dtype=ri.DT_BF16), 33), (dict(dtype=ri.DT_BF16, variant=2, chunk=16), 40)])
def test_transitions_over_the_8_bit_memory(sd, kw, T):
    """The oracle, given the memory as the library holds it, reads out the same logits."""
    import torch
    cfg = BASE.replace(**kw)
    model, oracle = _model(sd, cfg)
    st = sd.State(model, 2, T + 30, mem8=True)
    tok = _tokens(cfg, 2, T + 3)                                  # three encoded, not yet consumed
    st.encode(tok)
    mem, _ = _memory(sd, st, cfg)
    st.prefill(T)
    got = np.zeros((2, cfg.vocab), np.float32)
    st.readout(logits=got)
    st.check()
    for b in range(2):
        row = oracle.new_state()
        oracle.encode(row, tok[b])
        for g in range(cfg.groups):
            row.mem_k[g], row.mem_v[g] = (mem[g, b, w][:, :T + 3].transpose(1, 0, 2) for w in (0, 1))
        oracle.prefill(row, T)
        err = np.abs(got[b] - oracle.readout(row)).max()
        assert err <= tol_for(cfg), (b, err)
    # graph replays on a stream of its own: bit for bit the same
    twin = sd.State(model, 2, T + 30, mem8=True)
    s = torch.cuda.Stream()
    twin.encode(tok, stream=s)
    twin.prefill(T, stream=s)
    again = np.zeros_like(got)
    twin.readout(logits=again, stream=s)
    assert np.array_equal(got, again)


def test_bytes_of_an_8_bit_memory(sd):
    model, _ = _model(sd, BASE.replace(dtype=ri.DT_BF16))
    plain, eight = sd.State(model, 2, 256), sd.State(model, 2, 256, mem8=True)
    values = BASE.groups * 2 * BASE.heads * 256 * 64
    assert plain.bytes()[0] - eight.bytes()[0] == 2 * values - (values + BASE.groups * 2 * BASE.heads * 4 * 4)


def test_rows_restart_and_stand_at_unequal_positions(sd):
    """Packed documents over the 8-bit memory: each row as its last document alone."""
    model, _ = _model(sd, BASE)
    st = sd.State(model, 2, 100, mem8=True)
    tok = _tokens(BASE, 2, 90)
    starts = np.zeros((2, 90), np.uint8)
    starts[0, [0, 70]] = 1
    starts[1, [0, 3]] = 1
    st.prefill_packed(tok, starts)
    got = np.zeros((2, BASE.vocab), np.float32)
    st.readout(logits=got)
    for b, first in ((0, 70), (1, 3)):
        lone = sd.State(model, 1, 100, mem8=True)
        # the pieces of the packed run, so that pages meet the same tokens call by call
        cuts = [j for j in (3, 70, 90) if j > first]
        at = first
        for z in cuts:
            lone.encode(np.ascontiguousarray(tok[b:b + 1, at:z]))
            lone.prefill(z - at)
            at = z
        want = np.zeros((1, BASE.vocab), np.float32)
        lone.readout(logits=want)
        assert np.array_equal(got[b], want[0])


def _parts(sd, st, cfg, mem8):
    B, dh = st.batch, cfg.d // cfg.heads
    el = np.uint16 if cfg.dtype == ri.DT_BF16 else np.uint32
    pe, pd = st.positions()
    P = int(pe[0])
    out = {"s": st.read(sd.PART_S).reshape(B, -1),
           "e": st.read(sd.PART_E).view(np.uint32).reshape(B, st.max_len, -1)[:, int(pd[0]):P],
           "enc": st.read(sd.PART_ENC).view(el).reshape(B, -1, st.max_len, dh)[:, :, :P],
           "ring": st.read(sd.PART_RING).reshape(B, -1)}
    if cfg.variant == 2:
        out["R"] = st.read(sd.PART_R).reshape(B, -1)
    if mem8:
        n = -(-st.max_len // 64)
        used = -(-P // 64)
        out["mem"] = st.read(sd.PART_MEM).reshape(cfg.groups, B, n, -1)[:, :, :used].swapaxes(0, 1)
        out["scales"] = st.read(sd.PART_MEM_SCALES).reshape(cfg.groups, B, n, -1)[:, :, :used].swapaxes(0, 1)
    else:
        out["mem"] = st.read(sd.PART_MEM).view(el).reshape(B, -1, st.max_len, dh)[:, :, :P]
    return out


@pytest.mark.parametrize("mem8", [False, True])
@pytest.mark.parametrize("kw,shared", [(dict(), 0), (dict(variant=2, chunk=4, groups=1), 65),
                                       (dict(dtype=ri.DT_BF16, d=64, heads=1), 64), (dict(n_enc=0), 3)])
@pytest.mark.parametrize("host", [False, True])
def test_reorder_moves_all_that_a_row_needs(sd, mem8, kw, shared, host):
    import torch
    cfg = BASE.replace(**kw)
    model, _ = _model(sd, cfg)
    beams, B = 3, 6
    st = sd.State(model, B, 150, mem8=mem8)
    tok = _tokens(cfg, B, 75)
    tok[:, :shared] = np.repeat(tok[::beams, :shared], beams, 0)     # a search's rows share a prompt
    st.encode(tok)
    st.prefill(70)
    before = _parts(sd, st, cfg, mem8)
    parents = np.array([2, 0, 2, 1, 1, 0], np.int32)
    st.reorder(parents if host else torch.from_numpy(parents).cuda(), beams, shared)
    after = _parts(sd, st, cfg, mem8)
    source = parents + np.arange(B) // beams * beams
    for k in before:
        assert np.array_equal(after[k], before[k][source]), k
    # and the rows go on alike: same logits as a state fed the sources' tokens
    twin = sd.State(model, B, 150, mem8=mem8)
    twin.encode(np.ascontiguousarray(tok[source]))
    twin.prefill(70)
    a, b = np.zeros((B, cfg.vocab), np.float32), np.zeros((B, cfg.vocab), np.float32)
    for s, x in ((st, a), (twin, b)):
        s.prefill(5)
        s.encode(tok[:, :1].copy())
        s.step()
        s.readout(logits=x)
    assert np.array_equal(a, b)


def test_reorder_of_device_parents_out_of_range_leaves_rows(sd):
    import torch
    model, _ = _model(sd, BASE)
    st = sd.State(model, 4, 20)
    st.encode(_tokens(BASE, 4, 5))
    st.prefill(5)
    before = _parts(sd, st, BASE, False)
    st.reorder(torch.tensor([-1, 7, 1, 0], dtype=torch.int32, device="cuda"), 2)
    after = _parts(sd, st, BASE, False)
    for k in before:
        assert np.array_equal(after[k], before[k][[0, 1, 3, 2]]), k


@pytest.mark.parametrize("mem8", [False, True])
@pytest.mark.parametrize("kw,eos,temperature", [(dict(), -1, 1.0), (dict(variant=2, chunk=3), 2, 0.7),
                                                (dict(d=128, heads=1, groups=1), 0, 1.3)])
def test_beam_search_follows_the_oracle(sd, mem8, kw, eos, temperature):
    """Each step's choices are the best continuations by the oracle's own log-probabilities (to
    the fp32 tolerance), its scores theirs, and the rows afterwards the chosen sequences."""
    import torch
    cfg = BASE.replace(**kw)
    model, oracle = _model(sd, cfg, STD)
    G, K, prompt, steps = 2, 3, 62, 5
    B = G * K
    st = sd.State(model, B, 100, mem8=mem8)
    tok = np.repeat(_tokens(cfg, G, prompt), K, 0)
    st.encode(tok)
    st.prefill(prompt)
    scores = torch.full((G, K), -math.inf, device="cuda")
    scores[:, 0] = 0
    fin = torch.zeros(B, dtype=torch.uint8, device="cuda") if eos >= 0 else None
    par, new = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    seq = [list(tok[b]) for b in range(B)]
    at = scores.cpu().numpy().reshape(-1).astype(np.float64)
    done = np.zeros(B, bool)
    tol = tol_for(cfg)
    for _ in range(steps):
        logits = np.zeros((B, cfg.vocab), np.float32)
        st.readout(logits=logits)
        if not mem8:                                     # the logits themselves: the oracle's
            for b in range(B):
                row = oracle.new_state()
                oracle.encode(row, seq[b])
                oracle.prefill(row, len(seq[b]))
                # (the tolerance is that of weights of 0.02; the readout's are ten times those)
                assert np.abs(logits[b] - oracle.readout(row)).max() <= tol * STD / 0.02, b
        x = logits.astype(np.float64) / temperature
        x -= x.max(1, keepdims=True)
        x -= np.log(np.exp(x).sum(1, keepdims=True))
        st.beam_step(scores, par, new, K, finished=fin, eos=eos, temperature=temperature, shared=prompt)
        torch.cuda.synchronize()
        p, t, sc = par.cpu().numpy(), new.cpu().numpy(), scores.cpu().numpy().reshape(-1)
        f = fin.cpu().numpy().astype(bool) if eos >= 0 else np.zeros(B, bool)
        now, ended, grown = at.copy(), done.copy(), list(seq)
        for g in range(G):
            cand = at[g * K:(g + 1) * K, None] + x[g * K:(g + 1) * K]
            for k in range(K):
                if done[g * K + k]:
                    cand[k] = -math.inf
                    cand[k, eos] = at[g * K + k]
            order = np.argsort(-cand.reshape(-1), kind="stable")[:K]
            for i in range(K):
                r, q = g * K + i, int(p[g * K + i])
                assert (q, int(t[r])) == divmod(int(order[i]), cfg.vocab)
                now[r] = cand[q, t[r]]
                # one rounding to fp32 of a sum formed in fp64, from scores rounded the step before
                assert abs(sc[r] - now[r]) <= 2.0 ** -24 * abs(now[r]) + 1e-7
                ended[r] = done[g * K + q] or t[r] == eos
                grown[r] = seq[g * K + q] + [int(t[r])]
        at, done, seq = sc.astype(np.float64), ended, grown
        assert np.array_equal(done & (eos >= 0), f)
    pe, pd = st.positions()
    assert (pe == prompt + steps).all() and (pd == prompt + steps).all()
    # the rows' states are those of the chosen sequences
    got, want = np.zeros((B, cfg.vocab), np.float32), np.zeros((B, cfg.vocab), np.float32)
    st.readout(logits=got)
    twin = sd.State(model, B, 100, mem8=mem8)
    twin.encode(tok)
    twin.prefill(prompt)
    for j in range(prompt, prompt + steps):
        twin.encode(np.array([[s[j]] for s in seq], np.int32))
        twin.step()
    twin.readout(logits=want)
    assert np.array_equal(got, want)
    st.check()


def test_refusals(sd):
    import torch
    model, _ = _model(sd, BASE)
    assert sd.rlt_state_create_with(model.handle, 2, 8, 2)[0] == sd.RLT_E_ARG
    assert sd.rlt_state_create_with(model.handle, 0, 8, 1)[0] == sd.RLT_E_ARG
    small, _ = _model(sd, BASE.replace(heads=8))                  # heads of 16
    assert sd.rlt_state_create_with(small.handle, 2, 8, 1)[0] == sd.RLT_E_UNSUPPORTED
    st = sd.State(model, 4, 8, mem8=True)
    plain = sd.State(model, 4, 8)
    assert sd.rlt_state_read(plain.handle, sd.PART_MEM_SCALES)[0] == sd.RLT_E_UNSUPPORTED
    assert sd.rlt_state_save(st.handle, 0)[0] == sd.RLT_E_UNSUPPORTED
    snap = plain.save(0)
    assert sd.rlt_state_load(st.handle, 0, snap, snap.size) == sd.RLT_E_UNSUPPORTED
    par, tok = (torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(2))
    sc = torch.zeros(4, device="cuda")
    fin = torch.zeros(4, dtype=torch.uint8, device="cuda")

    def step(beams=2, state=st, scores=sc, finished=None, eos=-1, temperature=1.0, shared=0):
        return sd.rlt_beam_step(state.handle, scores, finished, eos, temperature, beams, shared, par, tok)

    for kw in (dict(beams=0), dict(beams=3), dict(beams=-1), dict(shared=-1), dict(temperature=0.0),
               dict(temperature=float("nan")), dict(eos=BASE.vocab), dict(finished=fin),
               dict(scores=np.zeros(4, np.float32)), dict(scores=None)):
        assert step(**kw) == sd.RLT_E_ARG, kw
    assert sd.rlt_state_reorder(st.handle, par, 3) == sd.RLT_E_ARG
    assert sd.rlt_state_reorder(st.handle, np.array([0, 2, 0, 1], np.int32), 2) == sd.RLT_E_ARG
    assert sd.rlt_state_reorder(st.handle, None, 2) == sd.RLT_E_ARG
    st.encode(_tokens(BASE, 4, 8))
    assert step() == sd.RLT_E_ORDER                              # tokens not yet consumed
    st.prefill(8)
    assert step() == sd.RLT_E_CAPACITY
    st.reset([1])
    assert step() == sd.RLT_E_ORDER                              # a search's rows at unequal positions
    assert sd.rlt_state_reorder(st.handle, par, 2) == sd.RLT_E_ORDER
    with pytest.raises(TypeError):
        st.beam_step(sc.double(), par, tok, 2)
    with pytest.raises(ValueError):
        st.reorder(par[:2], 2)
    # the state is as it was: row 0 goes on after a reset
    st.reset()
    st.encode(_tokens(BASE, 4, 2))
    st.prefill(2)
    assert step() == sd.RLT_OK
    torch.cuda.synchronize()
    st.check()
