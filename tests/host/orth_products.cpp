// How the products of an orthogonalisation are shared out, one line for each
// stack given on the command line as batch,rows,cols:
//   batch,rows,cols way product:tile,pair,deep,splits,whole,rest ...
// (the sharing rule of ecc_train_internal.hpp, compiled for the host).
#include <cstdio>

#include "ecc_train_internal.hpp"

using namespace ecc;

static void product(const char* name, int64_t rows, int64_t cols, int64_t batch, bool sym, int64_t k) {
  const OrthShare w = orth_share(rows, cols, batch, sym, (int)((k + 31) / 32));
  std::printf(" %s:%lld,%lld,%d,%d,%lld,%lld", name, (long long)w.tile, (long long)w.pair, (int)w.deep, w.splits,
              (long long)w.whole, (long long)w.rest);
}

int main(int argc, char** argv) {
  for (int i = 1; i < argc; ++i) {
    long long b, r, c;
    if (std::sscanf(argv[i], "%lld,%lld,%lld", &b, &r, &c) != 3) return 2;
    OrthArgs o{};
    o.batch = b;
    o.rows = r;
    o.cols = c;
    o.amplify = 1.0;  // five steps of the default coefficients stay below kMaxAmplify
    const OrthPlan p = orth_plan(b, r, c);
    std::printf("%lld,%lld,%lld %s", b, r, c, orth_is_thin(o) ? "thin" : orth_is_long(o) ? "long" : "direct");
    if (orth_is_long(o)) {
      product("last", p.mpad, p.npad, b, false, p.m);
    } else if (!orth_is_thin(o)) {
      product("gram", p.mpad, p.mpad, b, true, p.n);
      product("poly", p.mpad, p.mpad, b, true, p.m);
      product("update", p.mpad, p.npad, b, false, p.m);
      product("last", p.mpad, p.npad, b, false, p.m);
    }
    std::printf("\n");
  }
  return 0;
}
