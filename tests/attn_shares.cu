// Host model of an attention call's schedule, on the kernels' own arithmetic: reads calls from stdin and checks
// that the CTAs' segments cover every key tile of every item once, and that each part that is waited for is written.
//   rows_tile grid n_kv group few over B, then (rows, length) of each sequence
#include <cstdio>
#include <cstring>
#include <map>
#include <set>
#include <vector>

#include "tfq_attn.cuh"

using namespace tfq;

struct Call {
    int grid, n_kv, group, few, over;
    std::vector<SeqRows> q;
};

#define CHECK(x)                                                     \
    do {                                                             \
        if (!(x)) {                                                  \
            std::printf("call %d: %s does not hold\n", number, #x);  \
            return false;                                            \
        }                                                            \
    } while (0)

template <int ROWS, int KEYS, int kLeast, int kJoin>
bool check(const Call& call, int number)
{
    AttnParams p{};
    p.c.n_kv = call.n_kv;
    p.group = call.group;
    p.over = call.over;
    p.few = call.few != 0;
    p.B = (int)call.q.size();
    std::vector<SeqEntry> entries(p.B + 8);
    Shares<ROWS, KEYS, kLeast, kJoin> s(p, entries.data());
    int most = 0, sum = 0;
    for (const SeqRows& q : call.q) {
        const int2 c = s.counted(q);
        most = c.x > most ? c.x : most;
        sum += c.y;
    }
    if (kJoin > 0 && p.few && sum > 0)
        s.whole = s.whole_of(most, sum, call.grid);
    int64_t total = 0;
    for (int b = 0; b < p.B; ++b) {
        const SeqRows& q = call.q[b];
        entries[b] = SeqEntry{(int)total, q.r0, q.base, q.base >= 0 ? q.slot | q.rows << 16 : 0};
        total += q.base >= 0 ? s.all_units(q) : 0;
        CHECK(total < INT32_MAX);
    }
    s.total = (unsigned)total;
    s.deal(call.grid);
    CHECK(total == 0 || (s.ctas >= 1 && s.ctas <= (unsigned)call.grid));

    struct Item {
        int64_t next = 0;         // tiles so far, in order
        std::set<int> written;    // CTAs that write a part
        int c0 = -1, c1 = -1, tiles = 0;
    };
    std::map<std::vector<int>, Item> items;  // (sequence's first row, head, row tile)
    std::set<int> slots, owners;
    for (int cta = 0; cta < call.grid; ++cta) {
        const int u0 = s.start_of(cta), u1 = s.start_of(cta + 1);
        CHECK(u0 <= u1 && u1 <= total);
        for (int u = u0; u < u1;) {
            const Segment g = s.segment(u, u1);
            CHECK(g.units > 0);
            u += g.units;
            CHECK(g.t0 <= g.t1 && g.t1 <= g.nt && g.h < call.n_kv);
            if (g.t0 == g.t1)
                continue;
            Item& it = items[{g.q.r0, g.h, g.rt}];
            CHECK(it.next == g.t0);
            it.next = g.t1;
            it.tiles = g.nt;
            if (g.t0 == 0 && g.t1 == g.nt)
                continue;
            const int c0 = s.cta_of(g.first), c1 = s.cta_of(g.first + g.nt - 1);
            CHECK(c0 <= cta && cta <= c1 && c1 < call.grid);
            CHECK(it.c0 < 0 || (it.c0 == c0 && it.c1 == c1));
            it.c0 = c0;
            it.c1 = c1;
            CHECK((cta == c0) == (g.t0 == 0));               // the part that the joining CTAs read
            CHECK(slots.insert(2 * cta + (g.t0 == 0)).second);  // and that no other part lies in
            it.written.insert(cta);
        }
    }
    for (const SeqRows& q : call.q)
        for (int h = 0; q.base >= 0 && h < call.n_kv; ++h)
            for (int rt = 0; rt < s.row_tiles(q.rows); ++rt) {
                Item& it = items[{q.r0, h, rt}];
                CHECK(it.next == s.key_tiles(q.len()));
                CHECK(it.c0 < 0 || (int)it.written.size() == it.c1 - it.c0 + 1);
                CHECK(it.c0 < 0 || owners.insert(it.c0).second);  // its counters
            }
    return true;
}

int main()
{
    int number = 0, rows, B;
    Call c;
    while (std::scanf("%d %d %d %d %d %d %d", &rows, &c.grid, &c.n_kv, &c.group, &c.few, &c.over, &B) == 7) {
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
        const bool ok = rows == 16 ? check<16, 32, 8, 10>(c, number) : rows == 1616 ? check<16, 16, 8, 10>(c, number)
                      : rows == 32 ? check<32, 32, 8, 8>(c, number) : rows == 128 ? check<128, 64, 1, 0>(c, number)
                                                                                  : check<256, 64, 1, 0>(c, number);
        if (!ok)
            return 1;
        ++number;
    }
    std::printf("%d calls\n", number);
    return 0;
}
