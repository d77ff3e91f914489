"""The operators for long contexts as a server runs them together: rows are forked and extended, tokens appended with
scaled rotary positions, bounds updated, pages selected and attended over, the pool compacted; eagerly, captured into
graphs, and on streams of the caller's."""
import pytest

torch = pytest.importorskip("torch")
import long_ref as want  # noqa: E402
import paged_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
EPS_F16 = 2.0 ** -11


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_08_gb300 as m
    from exact_attention_forward_08_gb300 import _build
    _build.build()
    m.load_library()
    return m


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """A pool and its rows; every step's tensors come from the seed."""

    def __init__(self, fa, pages=200, heads=2, ratio=4, page=16, d=64, rows=6, width=24):
        self.fa, self.heads, self.ratio, self.page, self.d, self.rows, self.width = fa, heads, ratio, page, d, rows, width
        self.k = torch.zeros(pages, heads, page, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        self.v = torch.zeros_like(self.k)
        self.ks = torch.full((pages, heads), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
        self.vs = self.ks.clone()
        self.bounds = torch.zeros(pages, heads, 2, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.lens, self.refs = int32([0] * rows), int32([0] * pages)
        self.cos_sin = fa.rotary_table(width * page, d, scaling="by_parts", factor=4.0, original=64.0, high=8.0)

    def pool(self):
        return self.k, self.v, self.ks, self.vs

    def step(self, parents, new, seed, top=4):
        fa, g = self.fa, torch.Generator().manual_seed(seed)
        self.table, self.lens, self.refs = fa.kv_fork(int32(parents), *self.pool(), self.table, self.lens, self.refs,
                                                      new_tokens=int32(new), k_bounds=self.bounds)
        total = sum(new)
        cu = int32([sum(new[:b]) for b in range(self.rows + 1)])
        q = torch.randn(total, self.heads * self.ratio, self.d, generator=g).to(torch.bfloat16).cuda()
        k, v = (torch.randn(total, self.heads, self.d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        q = fa.kv_append(k, v, *self.pool(), self.table, self.lens, cu, q=q, cos_sin=self.cos_sin)
        fa.kv_bounds(self.k, self.bounds, self.table, self.lens, cu, total)
        lists, list_lens = fa.kv_select(q, self.bounds, self.ks, self.table, self.lens, cu, max(new), self.page, top, keep_first=1)
        o, lse = fa.attention_forward_lists(q, *self.pool(), lists, list_lens)
        return q, cu, lists, list_lens, o, lse

    def cpu_cache(self):
        """The pool as paged_ref describes one."""
        c = ref.Cache([1], self.heads, self.page, self.d, self.d)
        c.k, c.v, c.k_scale, c.v_scale = (t.cpu() for t in self.pool())
        c.num_pages, c.table, c.lens = self.k.shape[0], self.table.cpu(), self.lens.tolist()
        return c

    def check(self, q, cu, lists, list_lens, o, lse, top=4):
        torch.cuda.synchronize()
        code, detail = self.fa.fa_device_status()
        assert code == 0, (code, detail)
        c = self.cpu_cache()
        # the bounds are those of the codes, the lists those of the bounds, the results those of the lists
        full = want.all_bounds(c).float()
        for b, n in enumerate(c.lens):
            mine = c.table[b, :-(-n // self.page)].long()
            assert torch.equal(self.bounds.float().cpu()[mine], full[mine])
        ex, ex_lens = want.select(q.cpu(), self.bounds.cpu(), c.k_scale, c.table, c.lens, cu.tolist(), self.page, top, True, 1, 1)
        assert torch.equal(lists.long().cpu(), ex) and torch.equal(list_lens.long().cpu(), ex_lens)
        ref.check_attention(o, lse, want.lists_attention(q, c, lists, list_lens.tolist()), EPS_F16)
        # every page's count is the number of rows that hold it
        uses = [0] * c.num_pages
        for b, n in enumerate(c.lens):
            for p in c.table[b, :-(-n // self.page)].tolist():
                uses[p] += 1
        assert self.refs.tolist() == uses


STEPS = [([-1] * 6, [100, 37, 16, 1, 64, 90]), ([0, 1, 2, 3, 4, 5], [1, 1, 1, 1, 1, 1]), ([0, 0, 0, 1, 1, 5], [1, 2, 1, 1, 5, 1]),
         ([0, 1, 2, -1, 4, 5], [1, 1, 1, 70, 1, 1]), ([2, 2, 1, 3, 3, 0], [1, 1, 1, 1, 1, 1]), ([0, 1, 2, 3, 4, 5], [30, 1, 1, 2, 1, 1])]


def test_a_server_of_beams_and_requests(fa):
    s = Server(fa)
    for i, (parents, new) in enumerate(STEPS):
        out = s.step(parents, new, i)
        s.check(*out)
        if i in (2, 4):  # whatever was attended over is attended over alike when its pages have moved
            q, cu, lists, list_lens, o, lse = out
            s.table, s.refs, page_map, used = fa.kv_compact(*s.pool(), s.table, s.lens, s.refs, k_bounds=s.bounds)
            moved = torch.where(lists >= 0, page_map[lists.clamp(min=0).long()], lists)
            again, again_lse = fa.attention_forward_lists(q, *s.pool(), moved, list_lens)
            assert torch.equal(again, o) and torch.equal(again_lse, lse)
            assert int(used) == int((s.refs > 0).sum()) and not s.refs[int(used):].any()
            same = fa.kv_select(q, s.bounds, s.ks, s.table, s.lens, cu, max(new), s.page, 4, keep_first=1)[0]
            assert torch.equal(same, moved)


def test_all_pages_selected_is_the_whole_attention(fa):
    s = Server(fa)
    for i, (parents, new) in enumerate(STEPS[:3]):
        q, cu, lists, list_lens, o, lse = s.step(parents, new, i, top=24)
        c = s.cpu_cache()
        ref.check_attention(o, lse, ref.attention(q, c.k, c.v, c.k_scale, c.v_scale, c.table, c.lens, cu.tolist(), 16, True), EPS_F16)


def decode_graph(fa, s, q, k, v, cu, workspaces):
    """One captured decoding step of s.rows tokens that leaves its results where the next one finds them."""
    sel, att, pages = workspaces
    out = {}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        table, lens, refs = fa.kv_fork(s.parents, *s.pool(), s.table, s.lens, s.refs, new_tokens=s.ones, k_bounds=s.bounds,
                                       workspace=pages)
        rotated = fa.kv_append(k, v, *s.pool(), table, lens, cu, q=q, cos_sin=s.cos_sin)
        fa.kv_bounds(s.k, s.bounds, table, lens, cu, s.rows)
        lists, list_lens = fa.kv_select(rotated, s.bounds, s.ks, table, lens, cu, 1, s.page, 4, keep_first=1, workspace=sel)
        o, lse = fa.attention_forward_lists(rotated, *s.pool(), lists, list_lens, workspace=att)
        s.table.copy_(table)
        s.lens.copy_(lens)
        s.refs.copy_(refs)
    out.update(rotated=rotated, lists=lists, list_lens=list_lens, o=o, lse=lse)
    return graph, out


def test_captured_steps_that_share_workspaces(fa):
    """Two graphs over the same workspaces and cache, replayed by turns with new tokens and parents each time."""
    s = Server(fa)
    s.step(*STEPS[0], 0)
    s.parents, s.ones = int32(range(6)), int32([1] * 6)
    cu = int32(range(7))
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in
          (fa.fa_kv_select_workspace_size(6, 6, 2, s.width), fa.fa_fwd_lists_workspace_size(8, 2, 64),
           fa.fa_kv_pages_workspace_size(6, 6, 200))]
    tensors = [[torch.zeros(6, h, 64, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2)] for _ in range(2)]
    graphs = [decode_graph(fa, s, *t, cu, ws) for t in tensors]
    for i in range(6):
        graph, out = graphs[i % 2]
        g = torch.Generator().manual_seed(i)
        for t in tensors[i % 2]:
            t.copy_(torch.randn(t.shape, generator=g).to(torch.bfloat16))
        s.parents.copy_(int32([[0, 1, 2, 3, 4, 5], [0, 0, 0, 3, 3, 3], [1, 2, 3, 4, 5, 0]][i % 3]))
        graph.replay()
        s.check(out["rotated"], cu, out["lists"], out["list_lens"], out["o"], out["lse"])


def test_a_stream_of_the_callers(fa):
    """The whole step on a stream that is not the current one gives the same; what it allocates lives on that stream."""
    a, b = Server(fa), Server(fa)
    side = torch.cuda.Stream()
    for i, (parents, new) in enumerate(STEPS[:4]):
        plain = a.step(parents, new, i)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            inside = b.step(parents, new, i)
        side.synchronize()
        for x, y in zip(plain, inside):
            assert torch.equal(x, y)
    # and by argument
    q, cu, lists, list_lens, o, lse = plain
    torch.cuda.synchronize()
    got = fa.kv_select(q, a.bounds, a.ks, a.table, a.lens, cu, 70, 16, 4, keep_first=1, stream=side)
    res = fa.attention_forward_lists(q, *a.pool(), *got, stream=side)
    fork = fa.kv_fork(int32(range(6)), *a.pool(), a.table, a.lens, a.refs, stream=side)
    comp = fa.kv_compact(*a.pool(), a.table, a.lens, a.refs, stream=side)
    side.synchronize()
    assert torch.equal(got[0], lists) and torch.equal(got[1], list_lens) and torch.equal(res[0], o) and torch.equal(res[1], lse)
    assert torch.equal(fork[1], a.lens) and torch.equal(fork[2], a.refs)
    assert int(comp[3]) == int((a.refs > 0).sum())
    assert fa.fa_device_status()[0] == 0


def test_two_calls_at_once_with_their_own_workspaces(fa):
    """Selections and attentions of two caches on two streams, many times over, give what each gives alone."""
    servers = [Server(fa), Server(fa, pages=260, heads=1, ratio=20, page=32, d=128)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    alone = []
    for s in servers:
        s.step(*STEPS[0], 1)
        alone.append(s.step(*STEPS[1], 2))
    torch.cuda.synchronize()
    results = [[], []]
    for _ in range(20):
        for i, (s, stream) in enumerate(zip(servers, streams)):
            with torch.cuda.stream(stream):
                q, cu = alone[i][0], alone[i][1]
                lists, lens = fa.kv_select(q, s.bounds, s.ks, s.table, s.lens, cu, 1, s.page, 4, keep_first=1)
                results[i].append((lists, lens, *fa.attention_forward_lists(q, *s.pool(), lists, lens)))
    torch.cuda.synchronize()
    for i in range(2):
        for got in results[i]:
            for x, y in zip(got, alone[i][2:]):
                assert torch.equal(x, y)


def test_a_pool_of_more_than_four_gigabytes(fa):
    """The last pages of a pool whose offsets pass 32 bits: bounds, selection, attention, a fork's copy, a compaction."""
    heads, page, d, lens = 8, 128, 128, [300, 129]
    pages = 36000  # 4.7 GB of keys
    small = ref.Cache(lens, heads, page, d, d, spare=0)
    n = small.num_pages
    last = torch.arange(pages - n, pages)
    k, v = (torch.empty(pages, heads, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, heads), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    k[last], v[last] = small.k.view(torch.uint8).cuda(), small.v.view(torch.uint8).cuda()
    ks[last], vs[last] = small.k_scale.view(torch.uint8).cuda(), small.v_scale.view(torch.uint8).cuda()
    pool = (*(t.view(torch.float8_e4m3fn) for t in (k, v)), *(t.view(torch.float8_e8m0fnu) for t in (ks, vs)))
    table = torch.where(small.table >= 0, small.table + (pages - n), small.table).to(torch.int32).cuda()
    seqlens, refs = int32(lens), int32([0] * (pages - n) + [1] * n)
    bounds = torch.zeros(pages, heads, 2, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    cu = int32([0, 300, 429])
    fa.kv_bounds(pool[0], bounds, table, seqlens, cu, 429)
    full = want.all_bounds(small)
    assert torch.equal(bounds[pages - n:].float().cpu(), full.float())
    q = torch.randn(2, 16, d, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    one = int32([0, 1, 2])
    lists, list_lens = fa.kv_select(q.cuda(), bounds, pool[2], table, seqlens, one, 1, page, 2)
    ex, ex_lens = want.select(q, full, small.k_scale, small.table, lens, [0, 1, 2], page, 2)
    assert torch.equal(lists.cpu().long(), torch.where(ex >= 0, ex + pages - n, ex)) and torch.equal(list_lens.cpu().long(), ex_lens)
    o, lse = fa.attention_forward_lists(q.cuda(), *pool, lists, list_lens)
    ref.check_attention(o, lse, want.lists_attention(q, small, ex, ex_lens.tolist()), EPS_F16)
    # a copy from the last page to page 0, then all pages to the front
    table2, lens2, refs2 = fa.kv_fork(int32([0, 1, 1]), *pool, table, seqlens, refs, k_bounds=bounds)
    assert table2[2, 1] == 0 and lens2.tolist() == [300, 129, 129]
    assert torch.equal(k[0, :, :1], k[table2[1, 1].long(), :, :1]) and torch.equal(v[0, :, :1], v[table2[1, 1].long(), :, :1])
    table3, refs3, page_map, used = fa.kv_compact(*pool, table2, lens2, refs2, k_bounds=bounds)
    assert int(used) == n + 1 and int(table3.max()) == n
    moved = torch.where(lists >= 0, page_map[lists.clamp(min=0).long()], lists)
    again, again_lse = fa.attention_forward_lists(q.cuda(), *pool, moved, list_lens)
    assert torch.equal(again, o) and torch.equal(again_lse, lse)
    assert fa.fa_device_status()[0] == 0


def test_workspaces_go_back(fa):
    """Calls that allocate their own workspace leave nothing allocated, calls that are refused neither; inside a graph the
    memory is the graph's."""
    s = Server(fa)
    q, cu, lists, list_lens, o, lse = s.step(*STEPS[0], 0)
    outs = dict(table_out=torch.empty_like(s.table), refs_out=torch.empty_like(s.refs))
    parents, lens_out, page_map, used = int32(range(6)), torch.empty_like(s.lens), torch.empty_like(s.refs), int32([0])

    def calls(top=4, **kw):
        fa.kv_select(q, s.bounds, s.ks, s.table, s.lens, cu, 100, s.page, top, keep_first=1, lists=lists, list_lens=list_lens, **kw)
        fa.attention_forward_lists(q, *s.pool(), lists, list_lens, out=o, lse=lse, **kw)
        fa.kv_fork(parents, *s.pool(), s.table, s.lens, s.refs, seqlens_out=lens_out, **outs, **kw)
        fa.kv_compact(*s.pool(), s.table, s.lens, s.refs, page_map=page_map, used=used, **outs, **kw)

    side = torch.cuda.Stream()
    calls()
    torch.cuda.synchronize()
    want_o = o.clone()
    before = torch.cuda.memory_allocated()
    for i in range(50):
        calls(**({"stream": side} if i % 2 else {}))
        side.synchronize()
    with pytest.raises(fa.FaError):
        fa.attention_forward_lists(q, *s.pool(), lists, list_lens, scale=-1.0, out=o, lse=lse)
    with pytest.raises(fa.FaError):
        fa.kv_select(q, s.bounds, s.ks, s.table, s.lens, cu, 100, 48, 4, lists=lists, list_lens=list_lens)
    with pytest.raises(fa.FaError):
        fa.kv_fork(parents, *s.pool(), s.table, s.lens, s.refs, seqlens_out=s.lens, **outs)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() <= before
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    keep = torch.empty(1 << 22, dtype=torch.uint8, device="cuda").fill_(255)  # takes what the eager calls gave back
    o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want_o) and (keep == 255).all() and fa.fa_device_status()[0] == 0
