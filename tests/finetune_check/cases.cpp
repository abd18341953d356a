// The fine-tuning library on the CPU: every entry point called on buffers of
// exactly the size it may touch, each its own heap block, and its results
// compared with the formulas in double.  Built with AddressSanitizer and
// UndefinedBehaviorSanitizer, or with ThreadSanitizer, any access outside a
// buffer and any two threads on one LDS or global location without a barrier
// between them end the run.
//
//   cases [small]     small: the shapes that fit the thread checker's patience
//
// Prints "ok <cases> <launches>" and exits 0.
#define FINETUNE_WANT_GROUPS 8  // rows from which on a step holds them in registers, and below which they are split

#include "finetune_lib.hip"

#include <random>
#include <string>

namespace {

std::mt19937 gen(12345);
double uniform(double a, double b) { return std::uniform_real_distribution<double>(a, b)(gen); }
double normal() { return std::normal_distribution<double>()(gen); }
long cases = 0;

void require(bool ok, const std::string& what) {
  if (ok) return;
  std::fprintf(stderr, "FAILED: %s\n", what.c_str());
  std::exit(1);
}
void near(double got, double want, double tol, const std::string& what) {
  require(std::isnan(want) ? std::isnan(got) : std::fabs(got - want) <= tol * (1.0 + std::fabs(want)),
          what + ": got " + std::to_string(got) + " want " + std::to_string(want));
}

double load(const void* p, int64_t i, int dt) {
  if (dt == 0) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return dt == 1 ? finetune::Bf16::widen(h) : finetune::F16::widen(h);
}
void store(void* p, int64_t i, int dt, double v) {
  if (dt == 0)
    static_cast<float*>(p)[i] = static_cast<float>(v);
  else
    static_cast<uint16_t*>(p)[i] =
        dt == 1 ? finetune::Bf16::narrow(static_cast<float>(v)) : finetune::F16::narrow(static_cast<float>(v));
}
int bytes_of(int dt) { return dt == 0 ? 4 : 2; }
const double kTol[] = {3e-5, 2e-2, 3e-3};

// a heap block of exactly n elements, `skip` elements into it the first used one
struct Buf {
  char* base;
  int64_t n, skip;
  int dt;
  Buf(int64_t n_, int dt_, int64_t skip_ = 0) : n(n_ + skip_), skip(skip_), dt(dt_) {
    base = static_cast<char*>(std::malloc(static_cast<size_t>(n * bytes_of(dt)) + 1));
    std::memset(base, 0xff, static_cast<size_t>(n * bytes_of(dt)));
    base = static_cast<char*>(std::realloc(base, static_cast<size_t>(std::max<int64_t>(n * bytes_of(dt), 1))));
  }
  ~Buf() { std::free(base); }
  Buf(const Buf&) = delete;
  void* p() { return base + skip * bytes_of(dt); }
  float* f() { return static_cast<float*>(p()); }
  double operator[](int64_t i) { return load(p(), i, dt); }
  void set(int64_t i, double v) { store(p(), i, dt, v); }
};

void layer_norm_case(int64_t rows, int64_t d, int dt, int64_t pad, int64_t skip, bool in_place) {
  const std::string name = "layer_norm " + std::to_string(rows) + "x" + std::to_string(d) + " type " + std::to_string(dt);
  const int64_t xs = d + pad, span = rows ? (rows - 1) * xs + d : 0;
  Buf x(span, dt, skip), y(span, dt, skip), w(d, 0), b(d, 0), mean(rows, 0), rstd(rows, 0), dy(span, dt, skip),
      dx(span, dt, skip), dw(d, 0), db(d, 0);
  for (int64_t r = 0; r < rows; ++r)
    for (int64_t j = 0; j < d; ++j) {
      x.set(r * xs + j, 2.0 + normal());
      dy.set(r * xs + j, normal());
    }
  for (int64_t j = 0; j < d; ++j) {
    w.set(j, uniform(0.5, 1.5));
    b.set(j, normal());
  }
  require(layer_norm_fwd(x.p(), w.f(), b.f(), y.p(), mean.f(), rstd.f(), rows, d, xs, xs, 1e-5, dt, nullptr) == 0, name);
  std::vector<double> sw(d), sb(d);
  std::vector<std::vector<double>> want(rows, std::vector<double>(d));
  for (int64_t r = 0; r < rows; ++r) {
    double m = 0, v = 0;
    for (int64_t j = 0; j < d; ++j) m += x[r * xs + j] / d;
    for (int64_t j = 0; j < d; ++j) v += (x[r * xs + j] - m) * (x[r * xs + j] - m) / d;
    const double s = 1 / std::sqrt(v + 1e-5);
    near(mean[r], m, 1e-5, name + " mean");
    near(rstd[r] / s, 1.0, 1e-4, name + " rstd");
    double a = 0, c = 0;
    for (int64_t j = 0; j < d; ++j) {
      near(y[r * xs + j], (x[r * xs + j] - m) * s * w[j] + b[j], kTol[dt], name + " y");
      const double hat = (x[r * xs + j] - mean[r]) * rstd[r], g = dy[r * xs + j] * w[j];
      a += g / d;
      c += g * hat / d;
      sw[j] += dy[r * xs + j] * hat;
      sb[j] += dy[r * xs + j];
    }
    for (int64_t j = 0; j < d; ++j) {
      const double hat = (x[r * xs + j] - mean[r]) * rstd[r];
      want[r][j] = rstd[r] * (dy[r * xs + j] * w[j] - a - hat * c);
    }
  }
  int64_t need = 0;
  require(layer_norm_bwd_workspace(rows, d, &need) == 0, name);
  Buf ws(need / 4, 0);
  void* out = in_place ? dy.p() : dx.p();
  require(layer_norm_bwd(x.p(), w.f(), mean.f(), rstd.f(), dy.p(), out, dw.f(), db.f(), ws.p(), need, rows, d, xs, xs,
                         xs, dt, nullptr) == 0,
          name);
  for (int64_t j = 0; j < d; ++j) {
    near(dw[j], sw[j], 1e-4 * std::sqrt(static_cast<double>(rows + 1)), name + " dw");
    near(db[j], sb[j], 1e-4 * std::sqrt(static_cast<double>(rows + 1)), name + " db");
  }
  for (int64_t r = 0; r < rows; ++r)
    for (int64_t j = 0; j < d; ++j) near(load(out, r * xs + j, dt), want[r][j], 2 * kTol[dt], name + " dx");
  ++cases;
}

// logits in rows `pad` apart, labels with masked and (bad) unknown ones
struct LogitCase {
  int64_t n, t, v, ps, ss;
  int dt;
  Buf x, out;
  std::vector<int64_t> labels;
  finetune_logits in;
  finetune_dlogits grad;
  std::vector<double> lse, logp;
  LogitCase(int64_t n_, int64_t t_, int64_t v_, int dt_, int64_t pad, int64_t skip, bool bad)
      : n(n_), t(t_), v(v_), ps(v_ + pad), ss(t_ * (v_ + pad)), dt(dt_),
        x(n * t ? (n - 1) * ss + (t - 1) * ps + v : 0, dt, skip), out(n * t ? (n - 1) * ss + (t - 1) * ps + v : 0, dt, skip),
        labels(n * t), lse(n * t), logp(n * t) {
    for (int64_t r = 0; r < n * t; ++r) {
      labels[r] = uniform(0, 1) < 0.3 ? -100 : static_cast<int64_t>(uniform(0, 1) * v);
      if (bad && r == 1) labels[r] = v;
      if (bad && r == 2) labels[r] = -7;
      const int64_t at = r / t * ss + r % t * ps;
      double top = -1e300, sum = 0;
      for (int64_t j = 0; j < v; ++j) {
        x.set(at + j, 3 * normal());
        top = std::max(top, x[at + j]);
      }
      for (int64_t j = 0; j < v; ++j) sum += std::exp(x[at + j] - top);
      const bool known = labels[r] >= 0 && labels[r] < v;
      lse[r] = known ? top + std::log(sum) : labels[r] == -100 ? 0.0 : NAN;
      logp[r] = known ? x[at + labels[r]] - lse[r] : lse[r];
    }
    in = {x.p(), labels.data(), n, t, v, ss, ps, dt};
    grad = {out.p(), ss, ps};
  }
  void check_rows(Buf& gl, Buf& gp, const std::string& name) {
    for (int64_t r = 0; r < n * t; ++r) {
      near(gl[r], lse[r], 2e-5, name + " lse");
      near(gp[r], logp[r], 2e-5, name + " logp");
    }
  }
  void check_grad(void* p, const std::function<double(int64_t)>& g, const std::vector<double>& x0,
                  const std::string& name) {
    for (int64_t r = 0; r < n * t; ++r)
      for (int64_t j = 0; j < v; ++j) {
        const int64_t at = r / t * ss + r % t * ps + j;
        const bool known = labels[r] >= 0 && labels[r] < v;
        const double want = labels[r] == -100 ? 0.0
                            : known ? g(r) * ((j == labels[r] ? 1.0 : 0.0) - std::exp(x0[at] - lse[r]))
                                    : NAN;
        near(load(p, at, dt), want, kTol[dt], name + " dlogits");
      }
  }
  std::vector<double> values() {
    std::vector<double> q(x.n - x.skip);
    for (size_t i = 0; i < q.size(); ++i) q[i] = x[i];
    return q;
  }
};

void loss_case(int64_t n, int64_t t, int64_t v, int dt, int64_t pad, int64_t skip, bool in_place, bool bad) {
  const std::string name = "losses " + std::to_string(n) + "x" + std::to_string(t) + "x" + std::to_string(v) + " type " +
                           std::to_string(dt);
  LogitCase c(n, t, v, dt, pad, skip, bad);
  const std::vector<double> x0 = c.values();
  const int64_t rows = n * t;
  Buf logp(rows, 0), lse(rows, 0), ref(rows, 0), old(rows, 0), adv(n, 0), g(rows, 0);
  for (int64_t r = 0; r < rows; ++r) {
    ref.set(r, std::isfinite(c.logp[r]) ? c.logp[r] + 0.2 * normal() : 0.0);
    old.set(r, std::isfinite(c.logp[r]) ? c.logp[r] + 0.05 * normal() : 0.0);
    g.set(r, normal());
  }
  for (int64_t s = 0; s < n; ++s) adv.set(s, normal());
  int64_t need = 0;
  require(finetune_logits_workspace(&c.in, &need) == 0, name);
  Buf ws(need / 4, 0);
  const finetune_dlogits out = in_place ? finetune_dlogits{c.x.p(), c.ss, c.ps} : c.grad;
  const auto reset = [&]() {
    for (size_t i = 0; i < x0.size(); ++i) c.x.set(i, x0[i]);
  };

  require(token_logprob(&c.in, logp.f(), lse.f(), ws.p(), need, nullptr) == 0, name);
  c.check_rows(lse, logp, name);
  require(token_logprob_bwd(&c.in, lse.f(), g.f(), &out, nullptr) == 0, name);
  c.check_grad(out.data, [&](int64_t r) { return g[r]; }, x0, name + " logprob");
  reset();

  // policy: the step, then forward and backward
  Buf stats(2, 0), slope(rows, 0), stats2(2, 0), slope2(rows, 0), up(1, 0);
  for (int reduction = 0; reduction < 3; ++reduction) {
    const finetune_policy how{reduction, 0, 0.2, 0.3, 0.1};
    require(policy_loss_step(&c.in, old.f(), ref.f(), adv.f(), &how, 2.0, stats.f(), logp.f(), lse.f(), slope.f(), &out,
                             ws.p(), need, nullptr) == 0,
            name);
    c.check_rows(lse, logp, name);
    double total = 0, loss = 0, kl = 0;
    std::vector<double> count(n);
    for (int64_t r = 0; r < rows; ++r)
      if (c.labels[r] != -100) {
        total += 1;
        count[r / t] += 1;
      }
    std::vector<double> want(rows);
    for (int64_t r = 0; r < rows; ++r) {
      if (c.labels[r] == -100) continue;
      const double w = reduction == 0 ? 1 / total : reduction == 1 ? 1 / (count[r / t] * n) : 1;
      const double ratio = std::exp(c.logp[r] - old[r]), a = adv[r / t], q = ref[r] - c.logp[r];
      const double held = std::min(std::max(ratio, 0.8), 1.3) * a;
      loss += w * (-std::min(ratio * a, held) + 0.1 * (std::expm1(q) - q));
      kl += w * (std::expm1(q) - q);
      if (!std::isfinite(c.logp[r])) loss = kl = NAN;
      want[r] = w * ((ratio * a <= held ? -ratio * a : 0.0) - 0.1 * std::expm1(q));
    }
    near(stats[0], loss, 1e-4, name + " policy loss");
    near(stats[1], kl, 1e-4, name + " policy kl");
    c.check_grad(out.data, [&](int64_t r) { return 2 * want[r]; }, x0, name + " policy");
    reset();
    require(policy_loss_fwd(&c.in, old.f(), ref.f(), adv.f(), &how, stats2.f(), logp.f(), lse.f(), slope2.f(), ws.p(),
                            need, nullptr) == 0,
            name);
    near(stats2[0], loss, 1e-4, name + " policy loss forward");
    up.set(0, 2.0);
    require(policy_loss_bwd(&c.in, lse.f(), slope2.f(), up.f(), &out, nullptr) == 0, name);
    c.check_grad(out.data, [&](int64_t r) { return 2 * want[r]; }, x0, name + " policy backward");
    reset();
  }

  if (n % 2 == 0) {
    Buf loss(n / 2, 0), ratio(n, 0), sl(n, 0), dl(n / 2, 0);
    for (int kind = 0; kind < 3; ++kind) {
      const finetune_preference how{kind, kind == 1, 0.3, kind == 0 ? 0.1 : 0.0};
      require(preference_loss_step(&c.in, ref.f(), &how, 0.5, loss.f(), ratio.f(), logp.f(), lse.f(), sl.f(), &out, ws.p(),
                                   need, nullptr) == 0,
              name);
      c.check_rows(lse, logp, name);
      std::vector<double> lr(n), cnt(n), want(n);
      for (int64_t r = 0; r < rows; ++r)
        if (c.labels[r] != -100) {
          lr[r / t] += c.logp[r] - ref[r];
          cnt[r / t] += 1;
        }
      for (int64_t s = 0; s < n; ++s) {
        cnt[s] = how.average && cnt[s] > 0 ? cnt[s] : 1;
        lr[s] /= cnt[s];
        near(ratio[s], lr[s], 1e-4, name + " log-ratio");
      }
      for (int64_t b = 0; b < n / 2; ++b) {
        const double h = lr[b] - lr[b + n / 2], z = 0.3 * h, e = how.smoothing;
        const double l = kind == 0   ? (1 - e) * std::log1p(std::exp(-z)) + e * std::log1p(std::exp(z))
                         : kind == 1 ? (std::isnan(z) ? z : std::max(0.0, 1 - z))
                                     : (h - 0.5 / 0.3) * (h - 0.5 / 0.3);
        const double dh = kind == 0   ? -0.3 * ((1 - e) / (1 + std::exp(z)) - e / (1 + std::exp(-z)))
                          : kind == 1 ? (std::isnan(z) ? z : z < 1 ? -0.3 : 0.0)
                                      : 2 * (h - 0.5 / 0.3);
        near(loss[b], l, 1e-4, name + " preference loss");
        want[b] = dh / cnt[b];
        want[b + n / 2] = -dh / cnt[b + n / 2];
        dl.set(b, 0.5);
      }
      c.check_grad(out.data, [&](int64_t r) { return 0.5 * want[r / t]; }, x0, name + " preference");
      reset();
      require(preference_loss_fwd(&c.in, ref.f(), &how, loss.f(), ratio.f(), logp.f(), lse.f(), sl.f(), ws.p(), need,
                                  nullptr) == 0,
              name);
      require(preference_loss_bwd(&c.in, lse.f(), sl.f(), dl.f(), &out, nullptr) == 0, name);
      c.check_grad(out.data, [&](int64_t r) { return 0.5 * want[r / t]; }, x0, name + " preference backward");
      reset();
    }
  }
  ++cases;
}

// tensors of these sizes packed in one block at any element, clipped into another such block or in place
void clip_case(const std::vector<int64_t>& sizes, int64_t skip, int64_t out_skip, bool in_place, double max_norm) {
  const std::string name = "clip " + std::to_string(sizes.size()) + " tensors";
  int64_t total = 0;
  for (int64_t s : sizes) total += s;
  for (int dt = 0; dt < 3; ++dt) {
    Buf g(total, dt, skip), o(total, dt, out_skip), norm(1, 0);
    double sum = 0;
    for (int64_t i = 0; i < total; ++i) {
      g.set(i, normal());
      sum += g[i] * g[i];
    }
    std::vector<finetune_tensor> list;
    int64_t at = 0;
    for (int64_t s : sizes) {
      char* p = static_cast<char*>(g.p()) + at * bytes_of(dt);
      char* q = static_cast<char*>(o.p()) + at * bytes_of(dt);
      list.push_back({p, in_place ? p : q, s, dt});
      at += s;
    }
    std::vector<double> before(total);
    for (int64_t i = 0; i < total; ++i) before[i] = g[i];
    int64_t need = 0;
    require(grad_norm_workspace(list.data(), static_cast<int64_t>(list.size()), &need) == 0, name);
    Buf ws(need / 4, 0);
    require(grad_norm(list.data(), static_cast<int64_t>(list.size()), norm.f(), ws.p(), need, nullptr) == 0, name);
    near(norm[0], std::sqrt(sum), 1e-5, name + " norm");
    require(clip_grad_norm(list.data(), static_cast<int64_t>(list.size()), max_norm, 1e-6, norm.f(), ws.p(), need,
                           nullptr) == 0,
            name);
    near(norm[0], std::sqrt(sum), 1e-5, name + " norm");
    const double f = std::min(1.0, max_norm / (std::sqrt(sum) + 1e-6));
    for (int64_t i = 0; i < total; ++i) near(load(in_place ? g.p() : o.p(), i, dt), before[i] * f, kTol[dt], name);
  }
  ++cases;
}

}  // namespace

int main(int argc, char** argv) {
  const bool small = argc > 1 && std::string(argv[1]) == "small";
  for (int dt = 0; dt < 3; ++dt) {
    layer_norm_case(3, 5, dt, 2, 1, false);    // eight threads a row, cut pieces
    layer_norm_case(40, 128, dt, 0, 0, true);  // ... whole pieces, dx over dy
    layer_norm_case(5, 1000, dt, 3, 3, false);  // a wave a row
    layer_norm_case(0, 17, dt, 0, 0, false);
    loss_case(2, 1, 5, dt, 1, 1, false, false);  // a wave a row
    loss_case(2, 4, 150, dt, 7, 3, true, true);  // ... the rows held
    loss_case(3, 0, 9, dt, 0, 0, false, false);
    if (small && dt != 1) continue;
    loss_case(1, 2, 4300, dt, 1, 5, false, false);  // rows in parts
    layer_norm_case(2, 4093, dt, 1, 1, true);       // 256 threads a row
    if (small) continue;
    layer_norm_case(2, 1023, dt, 0, 0, true);
    layer_norm_case(2, 4096, dt, 0, 0, true);
    layer_norm_case(2, 5000, dt, 0, 0, false);  // 1024 threads a row
    layer_norm_case(2, 16383, dt, 0, 1, true);
    layer_norm_case(18, 16400, dt, 3, 1, true);  // the kernels of any length
    loss_case(2, 1, 9001, dt, 0, 3, true, false);
    loss_case(2, 32, 2100, dt, 1, 1, false, false);  // a wave a row of more pieces
    loss_case(2, 4, 4300, dt, 1, 1, true, false);    // rows held by 256 threads
    loss_case(2, 4, 20011, dt, 1, 1, false, false);  // ... by 512 and 1024
    loss_case(2, 4, 66000, dt, 0, 1, false, false);  // ... and past the widest in fp32
  }
  clip_case({5, 1, 0, 17}, 1, 1, false, 0.5);
  clip_case({9000, 3, 4096}, 3, 5, false, 1.0);
  clip_case({33, 8192, 7}, 2, 2, true, 1.0);
  clip_case({100, 50}, 0, 0, true, 1e9);
  std::vector<int64_t> many;
  for (int64_t i = 0; i < (small ? 240 : 300); ++i) many.push_back(i % 7);
  clip_case(many, 1, 1, false, 1.0);  // several tables
  std::printf("ok %ld %ld\n", cases, emu::launches);
  return 0;
}
