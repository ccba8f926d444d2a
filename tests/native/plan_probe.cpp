// Answers queries about the loss head's and Muon's host-side sizing (plan_xent.h,
// plan_muon.h) on stdin, one per line, so that they can be checked without a GPU:
//   fwd M K V pack  -> rows Kp Vc parts join_rows off_x off_w off_part off_run off_zt off_sum bytes
//   bwd M K V pack  -> rows both Kp Vc splits split_len acc off_row off_x off_w off_g off_acc bytes
//   bytes M K V     -> forward_bytes backward_bytes
//   muon batch K N  -> s sp Np tall parts one splits off_x0 off_x1 off_a off_b off_part off_sums bytes
//   tile batch I J R sym -> tile lower
#include "plan_muon.h"
#include "plan_xent.h"

#include <cstdio>
#include <cstring>

int main() {
    char op[16];
    long long a[5];
    while (std::scanf("%15s", op) == 1) {
        const int n = !std::strcmp(op, "tile") ? 5 : !std::strcmp(op, "bytes") || !std::strcmp(op, "muon") ? 3 : 4;
        for (int i = 0; i < n; ++i)
            if (std::scanf("%lld", a + i) != 1)
                return 2;
        if (!std::strcmp(op, "fwd")) {
            const auto f = lb::xent::forward(a[0], a[1], a[2], a[3] != 0);
            std::printf("%d %lld %lld %lld %d %lld %lld %lld %lld %lld %lld %lld\n", f.rows, (long long)f.Kp,
                        (long long)f.Vc, (long long)f.parts, f.join_rows, (long long)f.off_x, (long long)f.off_w,
                        (long long)f.off_part, (long long)f.off_run, (long long)f.off_zt, (long long)f.off_sum,
                        (long long)f.bytes);
        } else if (!std::strcmp(op, "bwd")) {
            const auto b = lb::xent::backward(a[0], a[1], a[2], a[3] != 0);
            std::printf("%d %d %lld %lld %d %lld %d %lld %lld %lld %lld %lld %lld\n", b.rows, b.both, (long long)b.Kp,
                        (long long)b.Vc, b.splits, (long long)b.split_len, (int)b.acc, (long long)b.off_row,
                        (long long)b.off_x, (long long)b.off_w, (long long)b.off_g, (long long)b.off_acc,
                        (long long)b.bytes);
        } else if (!std::strcmp(op, "bytes")) {
            std::printf("%lld %lld\n", (long long)lb::xent::forward_bytes(a[0], a[1], a[2]),
                        (long long)lb::xent::backward_bytes(a[0], a[1], a[2]));
        } else if (!std::strcmp(op, "muon")) {
            const auto p = lb::muon::plan(a[0], a[1], a[2]);
            std::printf("%lld %lld %lld %d %d %d %d %lld %lld %lld %lld %lld %lld %lld\n", (long long)p.s,
                        (long long)p.sp, (long long)p.Np, (int)p.tall, p.parts, p.one, p.splits, (long long)p.off_x0,
                        (long long)p.off_x1, (long long)p.off_a, (long long)p.off_b, (long long)p.off_part,
                        (long long)p.off_sums, (long long)p.bytes);
        } else if (!std::strcmp(op, "tile")) {
            const auto c = lb::muon::choose(a[0], a[1], a[2], a[3], a[4] != 0);
            std::printf("%d %d\n", (int)c.tile, (int)c.lower);
        } else {
            return 3;
        }
    }
    return 0;
}
