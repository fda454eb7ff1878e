// Host model of a prompt attention's schedule, on the kernel's own arithmetic: reads calls from stdin and checks that the
// CTAs' segments cover every key tile of every item once, and that each part that is waited for is written.
//   grid n_kv group over B, then (rows, length) of each sequence
#include <cstdio>
#include <map>
#include <set>
#include <vector>

#include "tfq_attn.cuh"

using namespace tfq;

#define CHECK(x)                                                    \
    do {                                                            \
        if (!(x)) {                                                 \
            std::printf("call %d: %s does not hold\n", number, #x); \
            return 1;                                               \
        }                                                           \
    } while (0)

int main()
{
    using S = PromptShares<128, 64, 2>;
    int number = 0, grid, n_kv, group, over, B;
    while (std::scanf("%d %d %d %d %d", &grid, &n_kv, &group, &over, &B) == 5) {
        AttnParams p{};
        p.c.n_kv = n_kv;
        p.group = group;
        p.over = over;
        p.B = B;
        std::vector<S::Entry> entries(B + 1);
        S s(p, entries.data());
        int64_t total = 0;
        int r0 = 0;
        for (int b = 0; b < B; ++b) {
            int rows, len;
            if (std::scanf("%d %d", &rows, &len) != 2)
                return 2;
            entries[b] = S::Entry{(int)total, r0, len - rows, rows};
            r0 += rows;
            total += s.all_units(len - rows, rows);
            CHECK(total < INT32_MAX);
        }
        s.total = (unsigned)total;
        s.deal(grid);
        struct Item {
            int next = 0, c0 = -1, c1 = -1;
            std::set<int> written;
        };
        std::map<std::vector<int>, Item> items;  // (sequence's first row, head, row tile)
        std::set<int> slots, owners;
        for (int cta = 0; cta < grid; ++cta) {
            const int u1 = s.start_of(cta + 1);
            for (int u = s.start_of(cta); u < u1;) {
                const Segment g = s.segment(u, u1);
                CHECK(g.units > 0 && g.t0 <= g.t1 && g.t1 <= g.nt && g.h < n_kv && g.rt < s.row_tiles(g.q.rows));
                u += g.units;
                if (g.t0 == g.t1)
                    continue;
                Item& it = items[{g.q.r0, g.h, g.rt}];
                CHECK(it.next == g.t0);
                it.next = g.t1;
                if (g.t0 == 0 && g.t1 == g.nt)
                    continue;
                const int c0 = s.cta_of(g.first), c1 = s.cta_of(g.first + g.nt - 1);
                CHECK(c0 <= cta && cta <= c1 && c1 < grid);
                CHECK(it.c0 < 0 || (it.c0 == c0 && it.c1 == c1));
                it.c0 = c0;
                it.c1 = c1;
                CHECK((cta == c0) == (g.t0 == 0));
                CHECK(slots.insert(2 * cta + (g.t0 == 0)).second);
                it.written.insert(cta);
            }
        }
        for (int b = 0; b < B; ++b)
            for (int h = 0; h < n_kv; ++h)
                for (int rt = 0; rt < s.row_tiles(entries[b].rows); ++rt) {
                    Item& it = items[{entries[b].r0, h, rt}];
                    const int last = ((rt + 1) * 128 - 1) / group;  // the tile's last row's token
                    const int len = entries[b].base + (last + 1 < entries[b].rows ? last + 1 : entries[b].rows);
                    CHECK(it.next == (len + 63) / 64);
                    CHECK(it.c0 < 0 || (int)it.written.size() == it.c1 - it.c0 + 1);
                    CHECK(it.c0 < 0 || owners.insert(it.c0).second);
                }
        ++number;
    }
    std::printf("%d calls\n", number);
    return 0;
}
