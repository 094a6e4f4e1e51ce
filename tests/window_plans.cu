// Prints how the library cuts the calls that its standard input names, one a line (the plans are functions of the sizes
// alone and need no GPU):  win Tq B Hq Hk D max_q max_k window sinks G Tp max_p
//                          few B Hq Hk D max_q max_k window sinks
//                          prefix_few B Hq Hk D max_q max_k max_p
//                          grad Tq Tk B Hq Hk D max_q max_k window sinks
#include <cstdio>
#include <cstring>

#include "window.h"

static void print(const vit::FewPlan &p)
{
    printf(" rows=%d row_tiles=%d chunk=%d n_split=%d room=%d partial_bytes=%zu", p.rows, p.row_tiles, p.chunk, p.n_split,
           p.room, p.partial_bytes);
}

int main()
{
    char kind[16];
    while (scanf("%15s", kind) == 1) {
        long long a[12];
        auto read = [&](int n) {
            for (int i = 0; i < n; ++i)
                if (scanf("%lld", &a[i]) != 1) return false;
            return true;
        };
        auto at = [&](int i) { return (int)a[i]; };
        if (!strcmp(kind, "win") && read(12)) {
            const vit::WinPlan p = vit::win_plan(a[0], at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), at(9), a[10], at(11));
            printf("apart=%d own_few=%d units=%d run_tiles=%d runs=%d max_items=%lld slots=%lld bytes=%zu", p.apart,
                   p.own_few, p.units, p.run_tiles, p.runs, (long long)p.max_items, (long long)p.slots, p.bytes);
            print(p.few);
        } else if (!strcmp(kind, "few") && read(8)) {
            printf("takes=%d", vit::window_takes_few(at(0), at(1), at(2), at(3), at(4), at(5), at(6), at(7)));
            print(vit::window_few_plan(at(0), at(1), at(2), at(3), at(4), at(5), at(6), at(7)));
        } else if (!strcmp(kind, "prefix_few") && read(7)) {
            printf("takes=%d", vit::prefix_takes_few(at(0), at(1), at(2), at(3), at(4), at(5), at(6)));
            print(vit::prefix_few_plan(at(0), at(1), at(2), at(3), at(4), at(5), at(6)));
        } else if (!strcmp(kind, "grad") && read(10)) {
            const vit::WinGradPlan p = vit::window_grad_plan(a[0], a[1], at(2), at(3), at(4), at(5), at(6), at(7), at(8), at(9));
            printf("lg_pack=%d max_dq=%lld max_dkv=%lld cut_over=%d run_tiles=%d max_cut=%d max_slots=%d bytes=%zu", p.lg_pack,
                   (long long)p.max_dq, (long long)p.max_dkv, p.cut_over, p.run_tiles, p.max_cut, p.max_slots, p.bytes);
        } else {
            return 1;
        }
        printf("\n");
    }
    return 0;
}
