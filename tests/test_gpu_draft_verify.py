"""Verification of drafted tokens on the GPU, through the package, against the
float64 reference.  The counts and tokens are whole numbers that comparisons
decide and must be equal; log p carries the fp32 rounding of the result and of
the sums it is formed from: 2^-20 absolute (sums of positive terms each good to
2^-22, and a logarithm below 40 rounded to 2^-19 at most is widened to 2^-18)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import draft_verify as dv

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import cross_entropy_tv_amd as lx  # noqa: E402
from _parity import announce  # noqa: E402

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TOL_LOGP = 2.0 ** -18
NINF = float("-inf")
DIRECT = 1 << 23  # up to this many positions times V the rows are summed in one step
ROOM = {"wide": False}


@pytest.fixture(params=[False, True], ids=["", "wide"], autouse=True)
def room(request):
    """Every test twice: as it is, and with room for so many drafts that a few sequences take the many ones' path."""
    ROOM["wide"] = request.param
    yield
    ROOM["wide"] = False


def rows(rng, n, V, scale=3.0):
    return torch.from_numpy(rng.standard_normal((n, V)).astype(np.float32) * np.float32(scale))


def on_device(t, dt, pad=0, offset=0):
    """A (n, V) device view of row stride V + pad whose first element lies `offset` elements into its buffer."""
    n, V = t.shape
    buf = torch.full((n * (V + pad) + offset + 8,), 77.0, dtype=dt, device=DEV)
    view = buf[offset:offset + n * (V + pad)].view(n, V + pad)[:, :V]
    view.copy_(t)
    return view


class Case:
    def __init__(self, seed, lens, V, dt="bf16", with_draft=True, temps=None, pad=(0, 0), offset=(0, 0), max_draft=None,
                 noise=0.7):
        rng = np.random.default_rng(seed)
        S, N = len(lens), sum(lens)
        self.lens, self.V, self.dt = lens, V, dt
        self.start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        self.max_draft = max(lens + [0]) if max_draft is None else max_draft
        if ROOM["wide"]:
            self.max_draft = max(self.max_draft, min(DIRECT // (S * V), 2 ** 20))  # (the most there is room for)
        z = rows(rng, N + S, V).to(DT[dt]).float()
        u = rows(rng, N, V, noise)
        for i in range(S):
            for j in range(lens[i]):
                u[self.start[i] + j] += z[self.start[i] + i + j]
        u = u.to(DT[dt]).float()
        self.z, self.u = z, (u if with_draft else None)
        self.temps = temps
        self.tokens = np.zeros(N, dtype=np.int64)
        for i in range(S):
            for j in range(lens[i]):
                k = self.start[i] + j
                t = 1.0 if temps is None else temps[i]
                if with_draft:
                    q = dv.probabilities(u[k].numpy(), t)
                    self.tokens[k] = dv.draw(q, rng.random())
                else:
                    self.tokens[k] = int(np.argmax(z[k + i].numpy())) if rng.random() < 0.8 else rng.integers(V)
        self.ua = rng.random(N).astype(np.float32)
        self.us = rng.random(S).astype(np.float32)
        self.pad, self.offset = pad, offset

    def reference(self):
        return dv.verify(self.z.numpy(), None if self.u is None else self.u.numpy(), self.tokens, self.start,
                         self.max_draft, self.temps, self.ua, self.us)

    def inputs(self):
        d = lambda a, t: torch.from_numpy(np.asarray(a, dtype=t)).to(DEV)  # noqa: E731
        return dict(target=on_device(self.z, DT[self.dt], self.pad[0], self.offset[0]),
                    draft=None if self.u is None else on_device(self.u, DT[self.dt], self.pad[1], self.offset[1]),
                    draft_tokens=d(self.tokens, np.int64), draft_start=d(self.start, np.int64),
                    max_draft=self.max_draft,
                    temperature=None if self.temps is None else d(self.temps, np.float32),
                    u_accept=d(self.ua, np.float32), u_sample=d(self.us, np.float32))

    def outputs(self):
        S, W = len(self.lens), self.max_draft + 1
        return (torch.full((S,), 99, dtype=torch.int64, device=DEV),
                torch.full((S, W), 99, dtype=torch.int64, device=DEV), torch.full((S, W), 99.0, device=DEV))

    def run(self, **kw):
        out = self.outputs()
        lx.lx_draft_verify(**self.inputs(), n_accepted=out[0], tokens=out[1], logprobs=out[2], **kw)
        torch.cuda.synchronize()
        return [o.cpu().numpy() for o in out]


def check(case, label):
    announce(f"draft_verify {label}")
    n, tok, lp = case.reference()
    gn, gtok, glp = case.run()
    assert np.array_equal(gn, n), f"{label}: accepted {gn} instead of {n}"
    assert np.array_equal(gtok, tok), f"{label}: tokens differ at {np.argwhere(gtok != tok)[:4]}"
    assert np.abs(glp - lp).max() <= TOL_LOGP, f"{label}: log p off by {np.abs(glp - lp).max()}"
    return n


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 1000, 2047, 2049, 8200, 50001])
@pytest.mark.parametrize("with_draft", [True, False], ids=["draft", "lookup"])
def test_vocabularies(V, dt, with_draft):
    check(Case(V, [3, 0, 5, 1, 4], V, dt, with_draft), f"V {V} {dt} draft {with_draft}")


@pytest.mark.parametrize("with_draft", [True, False], ids=["draft", "lookup"])
@pytest.mark.parametrize("lens", [[0], [1], [4], [0, 0, 0], [7, 0, 2] * 7, [1] * 70, [12, 3]],
                         ids=["0", "1", "4", "000", "ragged21", "70x1", "12+3"])
def test_batches(lens, with_draft):
    check(Case(5 + sum(lens), lens, 3001, "bf16", with_draft), f"lens {lens[:6]}")


def test_more_room_than_drafts():
    check(Case(8, [2, 0, 1], 513, max_draft=6), "max_draft 6 of 2")


@pytest.mark.parametrize("with_draft", [True, False], ids=["draft", "lookup"])
def test_temperatures_and_greedy(with_draft):
    temps = np.array([0.0, 0.25, 1.0, 3.0, 0.0, 1e-3, 1e-30, 50.0, -1.0], dtype=np.float32)
    check(Case(11, [4, 3, 2, 4, 0, 3, 3, 4, 2], 5003, "bf16", with_draft, temps=temps), "temperatures")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [((1, 0), (0, 0)), ((8, 3), (0, 5)), ((5, 5), (1, 2)), ((64, 64), (0, 0))])
def test_strides_and_alignments(pad, offset, dt):
    check(Case(13, [3, 5, 0, 2], 4099, dt, pad=pad, offset=offset), f"pad {pad} offset {offset}")


@pytest.mark.parametrize("V,S", [(151936, 1), (151936, 20), (262144, 3)])
def test_large_vocabularies(V, S):
    check(Case(17 + S, [4, 2, 5, 0][:S] * max(1, S // 4), V, "bf16"), f"{S} x {V}")


@pytest.mark.parametrize("with_draft", [True, False], ids=["draft", "lookup"])
def test_infinitely_hot(with_draft):
    """T = inf: every token that is not masked is as likely as any other."""
    V = 3000
    c = Case(71, [3, 0, 2], V, "f32", with_draft, temps=[1.0, 1.0, 1.0])
    c.z[:, 5:] = NINF
    if with_draft:
        c.u[:, 5:] = NINF  # p = q: all accepted
    c.tokens[:] = c.tokens % 5
    c.temps = [float("inf")] * 3
    c.ua[:] = 0.19 if not with_draft else 0.999
    announce(f"draft_verify infinitely hot {with_draft}")
    n, tok, lp = c.run()
    assert (n == c.lens).all()
    for i in range(3):
        assert (tok[i, :n[i]] == c.tokens[c.start[i]:c.start[i + 1]]).all() and tok[i, n[i]] == int(5 * c.us[i])
        assert np.abs(lp[i, :n[i] + 1] + np.log(5)).max() <= TOL_LOGP


def test_masked_vocabulary():
    """-inf and the type's lowest value on most of the vocabulary, in either row; rows with nothing left."""
    for dt in ("bf16", "f32", "f16"):
        c = Case(19, [3, 3, 2, 1, 2, 0, 1], 2500, dt)
        rng = np.random.default_rng(20)
        low = torch.finfo(DT[dt]).min
        keep = torch.from_numpy(rng.random(2500) < 0.05)
        c.z[:, ~keep] = NINF
        c.u[0:3, ~keep] = NINF
        c.z[4:7] = torch.where(keep, c.z[4:7], torch.tensor(low))
        c.u[3:6] = torch.where(keep, c.u[3:6], torch.tensor(low))
        at = np.flatnonzero(keep.numpy())
        c.tokens[:] = at[rng.integers(len(at), size=len(c.tokens))]
        c.tokens[1] = int(np.flatnonzero(~keep.numpy())[0])     # drafted, but masked in both rows
        s = c.start
        c.z[s[2] + 2] = NINF          # the first target row of sequence 2: nothing is accepted or drawn
        c.u[s[3]] = NINF              # the draft row of sequence 3: q = 0
        c.z[s[4] + 4 + 2] = NINF      # the row behind the last draft of sequence 4
        c.ua[s[4]:s[5]] = 0.0         # ... which is reached
        c.z[s[6] + 6] = low           # every logit the lowest value: a uniform row
        c.u[s[6]] = low
        c.ua[s[6]] = 0.999
        check(c, f"masked {dt}")


def test_rejections_that_leave_nothing():
    """Equal rows with a drafted token that neither can produce: drawn from p.  Without draft logits, a row whose
    only mass is the rejected token."""
    c = Case(23, [2, 2], 700, noise=0.0)
    c.z[:, 5] = NINF
    c.u[:, 5] = NINF
    c.tokens[:] = 5
    check(c, "equal rows, masked token")
    c = Case(24, [1, 1], 700, with_draft=False)
    c.z[0] = NINF
    c.z[0, 600] = 1.0
    c.tokens[0] = 600
    c.ua[0] = 1.0   # outside [0, 1), rejects even p = 1
    check(c, "the rejected token is all there is")


def test_tokens_outside_the_vocabulary():
    for with_draft in (True, False):
        c = Case(29, [2, 2, 2], 900, with_draft=with_draft)
        c.tokens[0], c.tokens[2], c.tokens[4] = -1, 900, 2 ** 40
        c.ua[:] = 0.0
        n = check(c, "outside")
        assert (n == 0).all()


def test_random_numbers_at_their_ends():
    for w in (0.0, float(np.nextafter(np.float32(1), np.float32(0))), 1.0):
        c = Case(31, [3, 0, 2], 3000)
        c.us[:] = w
        c.ua[:] = w
        check(c, f"all random numbers {w}")


@pytest.mark.parametrize("with_draft", [True, False], ids=["draft", "lookup"])
def test_comparisons_next_to_their_borders(with_draft):
    """r on either side of p / q, and w on either side of a border between two tokens, by one fp32 step."""
    for step in (-1, 1):
        c = Case(37, [1] * 24, 20000, "bf16", with_draft)
        for i in range(24):
            p = dv.probabilities(c.z[2 * i].numpy(), 1.0)
            x = int(c.tokens[i])
            q = dv.probabilities(c.u[i].numpy(), 1.0) if with_draft else None
            if i % 2 == 0:
                ratio = np.float32(min(p[x] / q[x] if with_draft else p[x], 0.99))
                c.ua[i] = np.nextafter(ratio, np.float32(2 if step > 0 else -2))
            else:
                c.ua[i] = 0.9999999  # mostly rejected: the draw of max(p - q, 0)
                mass = np.maximum(p - q, 0) if with_draft else np.where(np.arange(20000) == x, 0, p)
                sums = np.cumsum(mass)
                k = int(np.searchsorted(sums, 0.04 * i * sums[-1]))
                c.us[i] = np.nextafter(np.float32(sums[k] / sums[-1]), np.float32(2 if step > 0 else -2))
        check(c, f"borders {step}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_log_p_of_confident_tokens(dt):
    """p from 1/2 to 1 - 1e-6: log p keeps its relative precision, not only an absolute one.  It is -log(1 + rest),
    rest a sum of exponentials relative to the largest, each good to |a| 2^-24 + 2^-22 with a = log2 of it, below 30:
    2^-18 relative."""
    c = Case(59, [8] * 6, 20001, dt)
    for i in range(len(c.start) - 1):
        for j in range(8):
            z = c.z[c.start[i] + i + j]
            z[17 * i + j] = float(torch.logsumexp(z, 0)) + 2.0 * j
            c.u[c.start[i] + j] = z
            c.tokens[c.start[i] + j] = 17 * i + j
    c.z = c.z.to(DT[dt]).float()
    c.u = c.u.to(DT[dt]).float()
    c.ua[:] = 0.0
    n, tok, lp = c.reference()
    assert (n == 8).all() and (-lp[:, :8]).min() < 2e-6
    announce(f"draft_verify confident {dt}")
    _, gtok, glp = c.run()
    assert np.array_equal(gtok, tok)
    assert (np.abs(glp - lp)[:, :8] <= 2.0 ** -18 * np.abs(lp[:, :8])).all()


def test_sequences_that_do_not_fit_are_refused_alone():
    c = Case(41, [2, 2, 2, 2], 500)
    n, tok, lp = c.reference()
    for bad in ([0, 2, 1, 6, 8], [0, 2, 4, 9, 8], [0, 2, 8, 8, 8], [-3, 2, 4, 6, 8]):
        c2 = Case(41, [2, 2, 2, 2], 500)
        c2.start = np.array(bad, dtype=np.int64)
        announce(f"draft_verify starts {bad}")
        gn, gtok, glp = c2.run()
        for i in range(4):
            s, e = bad[i], bad[i + 1]
            if not (0 <= s <= e <= 8 and e - s <= c2.max_draft):
                assert gn[i] == -1 and (gtok[i] == -1).all() and (glp[i] == 0).all(), (bad, i)
            elif (s, e) == (c.start[i], c.start[i + 1]):
                assert gn[i] == n[i] and np.array_equal(gtok[i], tok[i]), (bad, i)


def test_without_logprobs_and_with_a_given_workspace():
    c = Case(43, [2, 3], 1234)
    n, tok, _ = c.reference()
    out = c.outputs()
    need = lx.lx_draft_verify_workspace_bytes(2, c.max_draft, 1234)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    lx.lx_draft_verify(**c.inputs(), n_accepted=out[0], tokens=out[1], logprobs=None, workspace=ws)
    assert np.array_equal(out[0].cpu().numpy(), n) and np.array_equal(out[1].cpu().numpy(), tok)
    assert (out[2] == 99.0).all()


def test_repeats_are_bitwise_equal_and_streams_are_kept():
    c = Case(47, [6, 5, 0, 3] * 8, 30001, "bf16")
    first = c.run()
    side = torch.cuda.Stream()
    for k in range(12):
        again = c.run(stream=side if k % 2 else None)
        for a, b in zip(first, again):
            assert np.array_equal(a.view(np.int32), b.view(np.int32))
    again = c.run(stream=side.cuda_stream)
    assert np.array_equal(first[1], again[1])


def test_captured_and_replayed():
    c = Case(53, [4, 0, 3, 2], 9001)
    a, out = c.inputs(), c.outputs()
    ws = torch.empty(lx.lx_draft_verify_workspace_bytes(4, c.max_draft, 9001), dtype=torch.uint8, device=DEV)
    call = lambda: lx.lx_draft_verify(**a, n_accepted=out[0], tokens=out[1], logprobs=out[2], workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    rng = np.random.default_rng(54)
    for _ in range(4):
        c.ua = rng.random(len(c.ua)).astype(np.float32)
        c.us = rng.random(len(c.us)).astype(np.float32)
        a["u_accept"].copy_(torch.from_numpy(c.ua))
        a["u_sample"].copy_(torch.from_numpy(c.us))
        for o in out:
            o.fill_(99)
        ws.fill_(0x5a)
        graph.replay()
        torch.cuda.synchronize()
        n, tok, lp = c.reference()
        assert np.array_equal(out[0].cpu().numpy(), n) and np.array_equal(out[1].cpu().numpy(), tok)
        assert np.abs(out[2].cpu().numpy() - lp).max() <= TOL_LOGP
        call()  # eager work between replays
        torch.cuda.synchronize()
        assert np.array_equal(out[1].cpu().numpy(), tok)


def test_loss_rejection_rate():
    """The emitted count's law next to the loss's own numbers: over many random numbers the share of rejected first
    drafts is the total variation distance of the two rows that lx_ce_tvd_forward gives."""
    V, S = 2000, 4096
    rng = np.random.default_rng(61)
    z, u = rows(rng, 1, V, 2.0), rows(rng, 1, V, 2.0)
    zt, ut = z.to(DEV).expand(2, V).contiguous(), u.to(DEV)
    f = lambda: torch.empty(1, device=DEV)  # noqa: E731
    ce, tvd, ls, lt, sg = f(), f(), f(), f(), f()
    lx.lx_ce_tvd_forward(ut, zt[:1], torch.zeros(1, dtype=torch.int64, device=DEV), -100, ce, tvd, ls, lt, sg)
    q = dv.probabilities(u[0].numpy(), 1.0)
    tok = np.searchsorted(np.cumsum(q), rng.random(S)).clip(max=V - 1)
    start = torch.arange(S + 1, device=DEV)
    n = torch.empty(S, dtype=torch.int64, device=DEV)
    out = torch.empty(S, 2, dtype=torch.int64, device=DEV)
    lx.lx_draft_verify(zt[:1].expand(2 * S, V).contiguous(), ut.expand(S, V).contiguous(),
                       torch.from_numpy(tok).to(DEV), start, 1, None, torch.rand(S, device=DEV),
                       torch.rand(S, device=DEV), n, out)
    # a share of 4096 Bernoulli draws: 5 standard deviations, 5 * sqrt(1 / 4 / 4096)
    assert abs(1.0 - n.double().mean().item() - tvd.item()) <= 5 * 0.5 / 64
