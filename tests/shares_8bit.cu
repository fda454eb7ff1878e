// Host model of the schedules over an 8-bit cache, on the kernels' own arithmetic: calls from stdin, every key tile of every
// item once, each part that is waited for written.
//   "A" and a call as attn_shares.cu has it: few rows, two CTAs an SM
//   "P" grid n_kv group over B, then (rows, length) of each sequence: prompts in row tiles of 256
#define main attn_shares_main
#include "attn_shares.cu"
#undef main

template <int ROWS>
bool check_prompt(const Call& call, int number)
{
    using S = PromptShares<ROWS, 64, 1>;
    AttnParams p{};
    p.c.n_kv = call.n_kv;
    p.group = call.group;
    p.over = call.over;
    p.B = (int)call.q.size();
    std::vector<typename S::Entry> entries(p.B + 1);
    S s(p, entries.data());
    int64_t total = 0;
    for (int b = 0; b < p.B; ++b) {
        const SeqRows& q = call.q[b];
        entries[b] = typename S::Entry{(int)total, q.r0, q.base, q.rows};
        total += s.all_units(q.base, q.rows);
        CHECK(total < INT32_MAX);
    }
    s.total = (unsigned)total;
    s.deal(call.grid);
    struct Item {
        int next = 0, c0 = -1, c1 = -1;
        std::set<int> written;
    };
    std::map<std::vector<int>, Item> items;  // (sequence's first row, head, row tile)
    std::set<int> slots, owners;
    for (int cta = 0; cta < call.grid; ++cta) {
        const int u1 = s.start_of(cta + 1);
        for (int u = s.start_of(cta); u < u1;) {
            const Segment g = s.segment(u, u1);
            CHECK(g.units > 0 && g.t0 <= g.t1 && g.t1 <= g.nt && g.h < call.n_kv && g.rt < s.row_tiles(g.q.rows));
            u += g.units;
            if (g.t0 == g.t1)
                continue;
            Item& it = items[{g.q.r0, g.h, g.rt}];
            CHECK(it.next == g.t0);
            it.next = g.t1;
            if (g.t0 == 0 && g.t1 == g.nt)
                continue;
            const int c0 = s.cta_of(g.first), c1 = s.cta_of(g.first + g.nt - 1);
            CHECK(c0 <= cta && cta <= c1 && c1 < call.grid);
            CHECK(it.c0 < 0 || (it.c0 == c0 && it.c1 == c1));
            it.c0 = c0;
            it.c1 = c1;
            CHECK((cta == c0) == (g.t0 == 0));
            CHECK(slots.insert(2 * cta + (g.t0 == 0)).second);
            it.written.insert(cta);
        }
    }
    for (const SeqRows& q : call.q)
        for (int h = 0; h < call.n_kv; ++h)
            for (int rt = 0; rt < s.row_tiles(q.rows); ++rt) {
                Item& it = items[{q.r0, h, rt}];
                const int last = ((rt + 1) * ROWS - 1) / call.group;  // the tile's last row's token
                const int seen = q.base + (last + 1 < q.rows ? last + 1 : q.rows);
                CHECK(it.next == (seen + 63) / 64);
                CHECK(it.c0 < 0 || (int)it.written.size() == it.c1 - it.c0 + 1);
                CHECK(it.c0 < 0 || owners.insert(it.c0).second);
            }
    return true;
}

int main()
{
    char kind;
    int number = 0, rows, B;
    Call c;
    while (std::scanf(" %c", &kind) == 1) {
        if (kind == 'A' ? std::scanf("%d %d %d %d %d %d %d", &rows, &c.grid, &c.n_kv, &c.group, &c.few, &c.over, &B) != 7
                        : std::scanf("%d %d %d %d %d", &c.grid, &c.n_kv, &c.group, &c.over, &B) != 5)
            return 2;
        c.q.assign(B, SeqRows{});
        int r0 = 0;
        for (SeqRows& q : c.q) {
            int len;
            if (std::scanf("%d %d", &q.rows, &len) != 2)
                return 2;
            q.r0 = r0;
            q.base = len - q.rows;
            r0 += q.rows;
        }
        if (!(kind == 'A' ? check<16, 32, 6, 10>(c, number) : check_prompt<256>(c, number)))
            return 1;
        ++number;
    }
    std::printf("%d calls\n", number);
    return 0;
}
