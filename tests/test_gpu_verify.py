"""verify_draft on the GPU against the oracle: whole numbers, so equal.  (All sums are of fp64 numbers;
a random number lies within their rounding of a border with probability 1e-12 or so.)"""
import numpy as np
import pytest

from oracle import msq_draft as T

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def msq():
    import block_wise_mixed_amd as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def inputs(rng, counts, V, chain, drawn, dtype, sharp=2.0):
    """Rows whose drafts are taken now and then: tokens from the drafter's distribution or its likeliest."""
    n = sum(counts)
    logits = rng.normal(size=(n, V)) * sharp
    near = logits + rng.normal(size=(n, V)) * 0.7
    target, draft = (torch.from_numpy(softmax(x)).to(dtype) for x in (logits, near))
    parents, tokens, at = [], [], 0
    for c in counts:
        used = {}
        for i in range(c):
            p = -1 if i == 0 else i - 1 if chain else int(rng.random() ** 1.5 * i)
            row = at + max(p, 0)
            if drawn:
                q = draft[row].double().numpy()
                tokens.append(int(rng.choice(V, p=q / q.sum())))
            else:
                k = used[p] = used.get(p, -1) + 1
                tokens.append(int(np.argsort(-near[row], kind="stable")[min(k, V - 1)]))
            parents.append(p)
        at += c
    return np.array(tokens), np.array(parents), target, draft, rng.random(n).astype(np.float32)


def check(msq, counts, tokens, parents, target, draft, uniform, chain=False, lead=0, **kw):
    """lead: rows before the first sequence and behind the last, outside both."""
    off = lead + np.concatenate([[0], np.cumsum(counts)]).astype(int)
    pad = lambda t: torch.cat([t.new_zeros((lead,) + t.shape[1:]), t, t.new_zeros((lead,) + t.shape[1:])]) if t is not None else None
    dev = lambda t: None if t is None else pad(torch.as_tensor(t)).cuda()
    ints = lambda t: None if t is None else dev(torch.as_tensor(t, dtype=torch.int32))
    token, taken, path = msq.verify_draft(ints(tokens), dev(target), i32(off), parents=None if chain else ints(parents),
                                          draft=dev(draft), uniform=dev(uniform), max_count=max(counts, default=0), **kw)
    torch.cuda.synchronize()
    token, taken, path = (t.cpu().numpy() for t in (token, taken, path))
    tn = target.double().numpy()
    dn = None if draft is None else draft.double().numpy()
    for b, n in enumerate(counts):
        sl = slice(off[b] - lead, off[b] - lead + n)
        want, rows = T.verify(tokens[sl], None if chain else parents[sl], tn[sl], None if dn is None else dn[sl],
                              None if uniform is None else uniform[sl])
        got = path[off[b]:off[b] + n]
        assert (token[b], taken[b], list(got)) == (want, len(rows), [off[b] + r for r in rows] + [-1] * (n - len(rows))), b
    return token, taken, path


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("way", ["drawn", "chosen", "largest"])
@pytest.mark.parametrize("chain", [True, False])
@pytest.mark.parametrize("V", [1, 2, 7, 1000, 1023, 5120, 32003])
def test_against_oracle(msq, V, chain, way, dtype):
    print("verify", V, chain, way, dtype, flush=True)
    rng = np.random.default_rng(V + chain)
    counts = [1, 5, 0, 26, 3, 64, 2] if V < 10000 else [5, 1, 12]
    tokens, parents, target, draft, u = inputs(rng, counts, V, chain, way == "drawn", dtype)
    draft = draft if way == "drawn" else None
    u = None if way == "largest" else u
    check(msq, counts, tokens, parents, target, draft, u, chain)
    check(msq, counts, tokens, parents, target, draft, u, chain, lead=3)


@pytest.mark.parametrize("way", ["drawn", "chosen", "largest"])
def test_many_sequences_and_one(msq, way):
    """Workgroups of a sequence from many to one, with numbers at every place of the distribution."""
    rng = np.random.default_rng(11)
    for B, V in ((1, 50000), (40, 3000), (700, 257)):
        print(way, B, V, flush=True)
        counts = [int(c) for c in rng.integers(1, 6, size=B)]
        tokens, parents, target, draft, u = inputs(rng, counts, V, False, way == "drawn", torch.float32, sharp=0.3)
        for k in range(3):
            check(msq, counts, tokens, parents, target, draft if way == "drawn" else None,
                  None if way == "largest" else u)
            u = rng.random(len(u)).astype(np.float32)


@pytest.mark.parametrize("drawn", [True, False])
def test_borders(msq, drawn):
    """Numbers at 0, 1, beyond and NaN; tokens outside the vocabulary; the same token among siblings;
    distributions with zeros, with nothing left, with nothing at all, not summing to one, with values
    that are no probabilities."""
    V, n = 600, 9
    rng = np.random.default_rng(5)
    for trial in range(60):
        p = softmax(rng.normal(size=(n, V)) * 3)
        q = softmax(rng.normal(size=(n, V)) * 3)
        p[rng.random((n, V)) < 0.5] = 0
        kind = trial % 6
        if kind == 1:
            p[:] = q                                    # nothing is left of p - q
        elif kind == 2:
            p[:] = 0
            p[:, 77] = 1                                # one token has it all
        elif kind == 3:
            p[0] = 0                                    # no distribution
        elif kind == 4:
            p *= 5
            p[:, ::7], p[:, 1::7], p[:, 2::7] = np.nan, -0.5, np.inf
            q[:, 3::7] = np.nan
        elif kind == 5:
            p[:] = 0
            p[:, [0, 3, V - 1]] = [0.5, 0.25, 0.25]
        parents = np.array([-1, 0, 0, 0, 1, 1, 4, 0, 0])
        tokens = np.array([0, 77, 77, 3, V - 1, 0, 3, -5, V + 3])
        u = np.array([[0, 1, 2.5, -1, np.nan][trial // 6 % 5]] + list(rng.choice([0, 1, -3, 7, np.nan, .5, .9], size=n - 1)), np.float32)
        check(msq, [n], tokens, parents, torch.from_numpy(p), torch.from_numpy(q) if drawn else None, u)


def test_siblings_one_after_another(msq):
    """Many siblings drawn from q, most of them not taken: what is left after each."""
    V, n = 2000, 40
    rng = np.random.default_rng(6)
    p, q = softmax(rng.normal(size=(n, V)) * 2), softmax(rng.normal(size=(n, V)) * 2)
    parents = np.array([-1] + [0] * (n - 1))
    for trial in range(8):
        tokens = rng.choice(V, size=n, p=q[0].astype(float) / q[0].astype(float).sum())
        u = rng.random(n).astype(np.float32)
        u[1:trial * 5] = 1.0
        check(msq, [n, 0, n], np.concatenate([tokens] * 2), np.concatenate([parents] * 2),
              torch.from_numpy(np.concatenate([p] * 2)), torch.from_numpy(np.concatenate([q] * 2)), np.concatenate([u, u[::-1].copy()]))
        check(msq, [n], tokens, parents, torch.from_numpy(p), None, u)


def test_largest_ties_and_logits(msq):
    """Equal largest entries, all entries equal, logits of any sign, infinities, rows of NaN."""
    V, n = 3001, 6
    rng = np.random.default_rng(7)
    x = rng.normal(size=(n, V)).astype(np.float32) * 10 - 50
    x[0, [5, 900, 3000]] = 7
    x[1] = -3
    x[2, 2999] = np.inf
    x[3] = -np.inf
    x[4] = np.nan
    x[4, 1234] = -8
    x[5] = np.nan
    tokens = np.array([0, 5, 0, 2999, 0, 1234])
    token, taken, path = check(msq, [n], tokens, np.arange(n) - 1, torch.from_numpy(x), None, None, chain=True)
    assert token[0] == -1 and taken[0] == n
    check(msq, [n], np.array([0, 900, 5, 1, 0, 2]), np.array([-1, 0, 0, 2, 2, 4]), torch.from_numpy(x), None, None)


def test_longest_sequences_and_strides(msq):
    rng = np.random.default_rng(8)
    tokens, parents, target, draft, u = inputs(rng, [1024, 3], 300, False, True, torch.float32)
    check(msq, [1024, 3], tokens, parents, target, draft, u)
    check(msq, [1024, 3], np.where(np.arange(1027) % 3 == 0, tokens, 0), parents, target, None, u, chain=True)
    # rows of a wider tensor, at an address that is no multiple of 16
    wide = torch.zeros(1027, 310).cuda()
    wide[:, 3:303] = target.cuda()
    a = msq.verify_draft(i32(tokens), wide[:, 3:303], i32([0, 1024, 1027]), parents=i32(parents),
                         uniform=torch.from_numpy(u).cuda(), max_count=1024)
    b = msq.verify_draft(i32(tokens), target.cuda(), i32([0, 1024, 1027]), parents=i32(parents),
                         uniform=torch.from_numpy(u).cuda(), max_count=1024)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    flipped = target.t().contiguous().t().cuda()
    c = msq.verify_draft(i32(tokens), flipped, i32([0, 1024, 1027]), parents=i32(parents),
                         uniform=torch.from_numpy(u).cuda(), max_count=1024)
    assert all(torch.equal(x, y) for x, y in zip(a, c))


def test_empty_calls(msq):
    for greedy in (False, True):
        u = None if greedy else torch.zeros(0, device="cuda")
        token, taken, path = msq.verify_draft(i32([]), torch.zeros(0, 50, device="cuda"), i32([0, 0, 0]), uniform=u)
        assert token.tolist() == [-1, -1] and taken.tolist() == [0, 0] and path.numel() == 0
        token, _, _ = msq.verify_draft(i32([]), torch.zeros(0, 50, device="cuda"), batch=0, uniform=u)
        assert token.numel() == 0


@pytest.mark.parametrize("greedy", [False, True])
def test_one_workspace_two_graphs_and_a_stream(msq, greedy):
    """Two captured calls that share a workspace, replayed in turn with new inputs and eager calls in
    between; the workspace holds anything before."""
    rng = np.random.default_rng(9)
    sizes = [([5] * 4, 9001), ([26, 3], 4000)]
    need = max(msq.verify_draft_workspace_bytes(sum(c), len(c), V, max(c), greedy) for c, V in sizes)
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
    states = []
    for counts, V in sizes:
        tokens, parents, target, draft, u = inputs(rng, counts, V, False, True, torch.float32)
        s = dict(tokens=i32(tokens), parents=i32(parents), target=target.cuda(), draft=draft.cuda(),
                 uniform=torch.from_numpy(u).cuda(), offset=i32(np.concatenate([[0], np.cumsum(counts)])), most=max(counts))
        s["call"] = lambda s=s, **kw: msq.verify_draft(s["tokens"], s["target"], s["offset"], parents=s["parents"],
                                                       draft=s["draft"], uniform=None if greedy else s["uniform"],
                                                       max_count=s["most"], **kw)
        s["call"](workspace=ws)
        torch.cuda.synchronize()
        s["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"]):
            s["out"] = s["call"](workspace=ws)
        states.append(s)
    side = torch.cuda.Stream()
    for step in range(6):
        for s in states:
            s["uniform"].copy_(torch.rand_like(s["uniform"]))
            s["target"].copy_(torch.softmax(2 * torch.randn_like(s["target"]), -1))
            torch.cuda.synchronize()
        for s in states:
            s["graph"].replay()
        torch.cuda.synchronize()
        for s in states:
            side.wait_stream(torch.cuda.current_stream())
            want = s["call"](stream=side)
            torch.cuda.current_stream().wait_stream(side)
            assert all(torch.equal(a, b) for a, b in zip(s["out"], want)), step


@pytest.mark.parametrize("greedy", [False, True])
def test_no_rows_in_the_workspace_of_more(msq, greedy):
    """A call without rows fits the workspace of calls with more of them (an empty tensor has no address, so
    nothing tells the two ways apart), and needs none itself."""
    B, V = 4, 32000
    ws = torch.empty(msq.verify_draft_workspace_bytes(20, B, V, greedy=greedy), dtype=torch.uint8, device="cuda")
    u = None if greedy else torch.zeros(0, device="cuda")
    for space in (ws, ws[:0]):
        for kw in (dict(offset=i32([0] * (B + 1))), dict(batch=B)):
            token, taken, path = msq.verify_draft(i32([]), torch.zeros(0, V, device="cuda"), uniform=u, workspace=space, **kw)
            assert token.tolist() == [-1] * B and taken.tolist() == [0] * B and path.numel() == 0


def test_siblings_of_nearly_the_target(msq):
    """A drafter that differs from the target by one unit of one entry and 1e-20 of another: what is left
    after the first sibling is 1e-20 in all, and every entry where both are equal has nothing."""
    V, n = 50, 6
    rng = np.random.default_rng(12)
    for trial in range(20):
        p = softmax(rng.normal(size=(1, V))).repeat(n, 0)
        q = p.copy()
        p[:, 1] = np.nextafter(q[:, 1], np.float32(0))
        p[:, 0], q[:, 0] = 1e-20, 0
        tokens = np.concatenate([[0, 1], rng.integers(2, V, size=n - 2)])
        u = np.concatenate([[rng.random()], np.ones(n - 1)]).astype(np.float32)
        token, taken, _ = check(msq, [n], tokens, np.array([-1] + [0] * (n - 1)), torch.from_numpy(p), torch.from_numpy(q), u)
        assert (token[0], taken[0]) == (0, 1)


@pytest.mark.parametrize("V", [2, 3, 8, 50, 9001])
def test_very_many_siblings(msq, V):
    """Some hundred siblings of one row, none taken: the entries that the target has most of beside the
    drafter stay, however small what was left of the first distribution has become.  In turn all of them
    below the first row, or half of them, then one that is taken, and the others below it."""
    n = 200
    rng = np.random.default_rng(V)
    for trial in range(8):
        p, q = softmax(rng.normal(size=(1, V)) * 2), softmax(rng.normal(size=(1, V)) * 2)
        if trial < 2:
            p[0], q[0] = np.eye(V)[0], 0.5 * np.eye(V)[0] + 0.5 * np.eye(V)[1]
        share = p[0] / np.maximum(q[0], 1e-9)
        tokens = np.full(n, int(np.argmin(share)))   # nothing is left of it from the first sibling on
        u = np.ones(n, np.float32)
        u[0] = rng.random()
        parents = np.array([-1] + [0] * (n - 1))
        if trial % 2:
            tokens[100], u[100] = int(np.argmax(share)), 0
            parents[101:] = 100
        _, taken, _ = check(msq, [n], tokens, parents, torch.from_numpy(p.repeat(n, 0)), torch.from_numpy(q.repeat(n, 0)), u)
        assert taken[0] == 1 + trial % 2


def test_largest_of_nothing_takes_no_token(msq):
    """Below a row of NaN no token is taken, whatever its number; nor one past the vocabulary elsewhere."""
    V = 700
    x = np.full((3, V), np.nan, np.float32)
    for t in (2 ** 31 - 1, -1, -2 ** 31, V, 0):
        token, taken, path = check(msq, [3], np.array([0, t, t]), np.array([-1, 0, 1]), torch.from_numpy(x), None, None)
        assert token[0] == -1 and taken[0] == 1
        check(msq, [3], np.array([0, t, t]), np.array([-1, 0, 1]), torch.from_numpy(np.nan_to_num(x)), None, None)
