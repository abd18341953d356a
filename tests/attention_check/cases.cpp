// The sublayer operators on the CPU: every entry point called on buffers of
// exactly the size it may touch, each its own heap block, and its results
// compared with the formulas in double.  Built with AddressSanitizer and
// UndefinedBehaviorSanitizer, or with ThreadSanitizer, any access outside a
// buffer and any two threads on one LDS or global location without a barrier
// between them end the run.  The borders of the position buckets are compared
// with whole-number arithmetic for every rule of a grid.
//
// Prints "ok <cases> <launches>" and exits 0.
#include "attention_lib.hip"
#include "attention_bf16.hip"
#include "attention_f16.hip"
#include "attention_f32.hip"

#include <random>
#include <string>

namespace {

std::mt19937 gen(4321);
double normal() { return std::normal_distribution<double>()(gen); }
long cases = 0;

void require(bool ok, const std::string& what) {
  if (ok) return;
  std::fprintf(stderr, "FAILED: %s\n", what.c_str());
  std::exit(1);
}
void near(double got, double want, double tol, const std::string& what) {
  require(got == want || std::fabs(got - want) <= tol * (1.0 + std::fabs(want)),
          what + ": got " + std::to_string(got) + " want " + std::to_string(want));
}

// a heap block of exactly n elements
struct Buf {
  int dt;
  char* base;
  Buf(int64_t n, int dt_) : dt(dt_) {
    base = static_cast<char*>(std::malloc(static_cast<size_t>(std::max<int64_t>(n * bytes(), 1))));
    std::memset(base, 0xff, static_cast<size_t>(n * bytes()));
  }
  ~Buf() { std::free(base); }
  Buf(const Buf&) = delete;
  int bytes() const { return dt == 0 ? 4 : 2; }
  float* f() { return reinterpret_cast<float*>(base); }
  double operator[](int64_t i) const {
    if (dt == 0) return reinterpret_cast<const float*>(base)[i];
    const uint16_t h = reinterpret_cast<const uint16_t*>(base)[i];
    return dt == 1 ? finetune::Bf16::widen(h) : finetune::F16::widen(h);
  }
  void set(int64_t i, double v) {
    const float x = static_cast<float>(v);
    if (dt == 0)
      f()[i] = x;
    else
      reinterpret_cast<uint16_t*>(base)[i] = dt == 1 ? finetune::Bf16::narrow(x) : finetune::F16::narrow(x);
  }
};
const double kTol[] = {5e-5, 3e-2, 5e-3};

int bucket_of(int64_t rel, const attention_buckets& b) {  // by whole powers, in long double where they are exact enough
  const int64_t side = b.two_sided ? b.count / 2 : b.count, small = side / 2, rest = side - small;
  const int64_t base = b.two_sided && rel > 0 ? side : 0, n = b.two_sided ? std::llabs(rel) : std::max<int64_t>(-rel, 0);
  if (n < small) return static_cast<int>(base + n);
  int64_t m = 0;
  const long double x = std::log(static_cast<long double>(n) / small), unit = std::log(static_cast<long double>(b.max_distance) / small);
  while (m + 1 < rest && x * rest >= unit * (m + 1) - 1e-13L) ++m;
  return static_cast<int>(base + small + m);
}

void bucket_rules() {
  for (int64_t two = 0; two < 2; ++two)
    for (int64_t side : {2, 3, 4, 5, 8, 16, 31, 64, 100, 256})
      for (int64_t distance : {2, 3, 8, 20, 64, 128, 300, 777, 1024}) {
        const attention_buckets b{two ? 2 * side : side, distance, two};
        if (finetune::check_buckets(&b) != RDFFT_OK) continue;
        const finetune::Buckets r = finetune::buckets_of(b);
        for (int64_t rel = -2100; rel <= 2100; ++rel)
          require(r.of(static_cast<int>(rel)) == bucket_of(rel, b),
                  "bucket of " + std::to_string(rel) + " among " + std::to_string(b.count) + " to " + std::to_string(distance));
        for (int c = 0; c < r.count; ++c) {
          int lo, hi;
          r.range(c, 2100, lo, hi);
          for (int rel = -2100; rel <= 2100; ++rel)
            require((r.of(rel) == c) == (rel >= lo && rel <= hi), "range of bucket " + std::to_string(c));
        }
      }
}

// tokens x heads x d, `pad` elements between heads
struct Rows {
  int64_t b, t, h, d, pad;
  Buf buf;
  Rows(int64_t b_, int64_t t_, int64_t h_, int64_t d_, int64_t pad_, int dt)
      : b(b_), t(t_), h(h_), d(d_), pad(pad_), buf(b * t * h ? (b * t * h - 1) * (d + pad) + d : 0, dt) {}
  int64_t at(int64_t i, int64_t j, int64_t k, int64_t x) const { return ((i * t + j) * h + k) * (d + pad) + x; }
  double operator()(int64_t i, int64_t j, int64_t k, int64_t x) const { return buf[at(i, j, k, x)]; }
  void fill() {
    for (int64_t i = 0; i < b * t * h; ++i)
      for (int64_t x = 0; x < d; ++x) buf.set(i * (d + pad) + x, normal());
  }
  attention_tensor arg() { return {buf.base, t * h * (d + pad), h * (d + pad), d + pad}; }
};

void attention_case(int64_t b, int64_t tq, int64_t tk, int64_t h, int64_t hk, int64_t d, int dt, bool causal, bool spans,
                    bool biased, int64_t pad) {
  const std::string name = "attention " + std::to_string(b) + "x" + std::to_string(tq) + "x" + std::to_string(tk) + "x" +
                           std::to_string(h) + "/" + std::to_string(hk) + "x" + std::to_string(d) + " type " +
                           std::to_string(dt);
  std::fprintf(stderr, "%s\n", name.c_str());
  Rows q(b, tq, h, d, pad, dt), k(b, tk, hk, d, pad, dt), v(b, tk, hk, d, 0, dt), o(b, tq, h, d, pad, dt),
      go(b, tq, h, d, 0, dt), dq(b, tq, h, d, pad, dt), dk(b, tk, hk, d, 0, dt), dv(b, tk, hk, d, pad, dt);
  for (Rows* r : {&q, &k, &v, &go}) r->fill();
  std::vector<int32_t> lo(b, 0), hi(b, static_cast<int32_t>(tk));
  if (spans)
    for (int64_t i = 0; i < b; ++i) lo[i] = static_cast<int32_t>(i), hi[i] = static_cast<int32_t>(i + 1 == b ? 0 : tk - 2 * i);
  const attention_buckets rule{6, 12, 1};
  Buf table(rule.count * h, 0), dtable(rule.count * h, 0), lse(b * h * tq, 0);
  for (int64_t i = 0; i < rule.count * h; ++i) table.set(i, normal());
  attention_problem a{b, tq, tk, h, hk, d, dt, 0.3, causal, spans ? lo.data() : nullptr, spans ? hi.data() : nullptr,
                      biased ? table.f() : nullptr, rule};
  const attention_tensor tq_ = q.arg(), tk_ = k.arg(), tv = v.arg(), to = o.arg(), tg = go.arg(), tdq = dq.arg(),
                         tdk = dk.arg(), tdv = dv.arg();
  int64_t need = 0;
  require(attention_workspace(&a, 0, &need) == 0, name);
  {
    Buf ws(need / 4, 0);
    require(attention_fwd(&a, &tq_, &tk_, &tv, &to, lse.f(), ws.base, need, nullptr) == 0, name);
  }
  require(attention_workspace(&a, 1, &need) == 0, name);
  {
    Buf ws(need / 4, 0);
    require(attention_bwd(&a, &tq_, &tk_, &tv, &to, lse.f(), &tg, &tdq, &tdk, &tdv, biased ? dtable.f() : nullptr,
                          ws.base, need, nullptr) == 0,
            name);
  }
  std::vector<double> wk(b * tk * hk * d), wv(b * tk * hk * d), wt(rule.count * h);
  for (int64_t i = 0; i < b; ++i)
    for (int64_t n = 0; n < h; ++n)
      for (int64_t r = 0; r < tq; ++r) {
        const int64_t m = n / (h / hk), last = causal ? std::min<int64_t>(hi[i], r + tk - tq + 1) : hi[i];
        std::vector<double> p(tk), dp(tk);
        double top = -INFINITY, sum = 0, delta = 0;
        for (int64_t j = lo[i]; j < last; ++j) {
          for (int64_t x = 0; x < d; ++x) p[j] += 0.3 * q(i, r, n, x) * k(i, j, m, x), dp[j] += go(i, r, n, x) * v(i, j, m, x);
          if (biased) p[j] += table[bucket_of(j - (r + tk - tq), rule) * h + n];
          top = std::max(top, p[j]);
        }
        for (int64_t j = lo[i]; j < last; ++j) sum += std::exp(p[j] - top);
        near(lse[(i * h + n) * tq + r], last > lo[i] ? top + std::log(sum) : -INFINITY, 1e-4, name + " lse");
        std::vector<double> wo(d), wq(d);
        for (int64_t j = lo[i]; j < last; ++j) p[j] = std::exp(p[j] - top) / sum, delta += p[j] * dp[j];
        for (int64_t j = lo[i]; j < last; ++j) {
          const double ds = p[j] * (dp[j] - delta);
          if (biased) wt[bucket_of(j - (r + tk - tq), rule) * h + n] += ds;
          for (int64_t x = 0; x < d; ++x) {
            wo[x] += p[j] * v(i, j, m, x);
            wq[x] += 0.3 * ds * k(i, j, m, x);
            wk[((i * tk + j) * hk + m) * d + x] += 0.3 * ds * q(i, r, n, x);
            wv[((i * tk + j) * hk + m) * d + x] += p[j] * go(i, r, n, x);
          }
        }
        for (int64_t x = 0; x < d; ++x) {
          near(o(i, r, n, x), wo[x], kTol[dt], name + " o");
          near(dq(i, r, n, x), wq[x], kTol[dt], name + " dq");
        }
      }
  for (int64_t i = 0; i < b * tk * hk; ++i)
    for (int64_t x = 0; x < d; ++x) {
      near(dk(i / hk / tk, i / hk % tk, i % hk, x), wk[i * d + x], 2 * kTol[dt], name + " dk");
      near(dv(i / hk / tk, i / hk % tk, i % hk, x), wv[i * d + x], 2 * kTol[dt], name + " dv");
    }
  if (biased)
    for (int64_t i = 0; i < rule.count * h; ++i) near(dtable[i], wt[i], 2e-3, name + " dbias");
  ++cases;
}

void bias_case(int64_t b, int64_t h, int64_t tq, int64_t tk, int dt, const attention_buckets& rule) {
  const std::string name = "bias " + std::to_string(tq) + "x" + std::to_string(tk) + " type " + std::to_string(dt);
  std::fprintf(stderr, "%s\n", name.c_str());
  Buf table(rule.count * h, 0), bias(h * tq * tk, dt), d(b * h * tq * tk, dt), dt_(rule.count * h, 0);
  for (int64_t i = 0; i < rule.count * h; ++i) table.set(i, normal());
  for (int64_t i = 0; i < b * h * tq * tk; ++i) d.set(i, normal());
  require(relative_bias_fwd(table.f(), bias.base, h, tq, tk, &rule, dt, nullptr) == 0, name);
  int64_t need = 0;
  require(relative_bias_workspace(b, h, tq, tk, &rule, &need) == 0, name);
  Buf ws(need / 4, 0);
  require(relative_bias_bwd(d.base, h * tq * tk, tq * tk, tk, dt_.f(), b, h, tq, tk, &rule, ws.base, need, dt, nullptr) == 0,
          name);
  std::vector<double> want(rule.count * h);
  for (int64_t n = 0; n < h; ++n)
    for (int64_t i = 0; i < tq; ++i)
      for (int64_t j = 0; j < tk; ++j) {
        const int c = bucket_of(j - (i + tk - tq), rule);
        near(bias[(n * tq + i) * tk + j], table[c * h + n], kTol[dt], name + " bias");
        for (int64_t m = 0; m < b; ++m) want[c * h + n] += d[((m * h + n) * tq + i) * tk + j];
      }
  for (int64_t i = 0; i < rule.count * h; ++i) near(dt_[i], want[i], 1e-3, name + " dtable");
  ++cases;
}

void dropout_case(int64_t rows, int64_t d, int64_t pad, int dt, bool residual) {
  const std::string name = "dropout " + std::to_string(rows) + "x" + std::to_string(d) + " type " + std::to_string(dt);
  std::fprintf(stderr, "%s\n", name.c_str());
  const int64_t n = (rows - 1) * (d + pad) + d;
  Buf x(n, dt), r(n, dt), y(n, dt);
  for (int64_t i = 0; i < n; ++i) x.set(i, 1.0 + 0.1 * normal()), r.set(i, normal());
  uint64_t seed = 5;
  const attention_dropout how{0.25, 2, 9, &seed};
  require(dropout_fwd(x.base, residual ? r.base : nullptr, y.base, rows, d, d + pad, d + pad, d + pad, &how, dt, nullptr) == 0,
          name);
  for (int64_t i = 0; i < rows * d; ++i) {
    const finetune::Philox g(static_cast<uint64_t>(i / 8), 9, 7);
    const int64_t at = i / d * (d + pad) + i % d;
    const double kept = g.bits(i % 8) >= 16384 ? x[at] * (4.0 / 3.0) : 0.0;
    near(y[at], kept + (residual ? r[at] : 0.0), kTol[dt], name);
  }
  ++cases;
}

}  // namespace

int main() {
  bucket_rules();
  for (int dt = 0; dt < 3; ++dt) {
    dropout_case(1, 37, 0, dt, true);
    dropout_case(5, 13, 3, dt, dt == 1);
    bias_case(dt + 1, 1, 7, 21 + dt, dt, {6, 12, 1});
    bias_case(2, 1, 3, 600, dt, {5, 9, 0});
  }
  attention_case(2, 5, 40, 2, 1, 5, 0, false, true, true, 1);
  attention_case(1, 70, 40, 1, 1, 16, 1, true, false, true, 0);
  attention_case(2, 40, 70, 2, 1, 40, 2, true, true, false, 8);
  attention_case(1, 2, 140, 2, 2, 9, 1, true, false, false, 3);  // the keys split over workgroups
  std::printf("ok %ld %ld\n", cases, emu::launches);
  return 0;
}
