// The launch rules of the fine-tuning library, on the host alone: for batches of
// every shape the C ABI admits, the kernel that holds a row a workgroup is
// chosen only where its launch stays below HIP's 2^32 threads, and is chosen
// where it should be.  Nothing is launched.
#include "finetune_lib.hip"

int main() {
  using namespace finetune;
  long held = 0, checks = 0;
  for (int64_t dt = 0; dt < 3; ++dt)
    for (int64_t vocab : {1, 7, 16, 100, 2051, 4096, 4104, 8200, 16391, 32776, 65536, 65540, 131072, 131080, 1 << 24})
      for (int shift = 0; shift < 32; ++shift)
        for (int64_t off : {-1, 0, 1}) {
          const int64_t rows = (int64_t(1) << shift) + off;
          if (rows < 1 || rows > 0x7fffffff) continue;
          const finetune_logits in{nullptr, nullptr, 1, rows, vocab, 0, vocab, dt};
          if (check_logits_dims(&in) != RDFFT_OK) return 2;
          int64_t threads = 0, pieces = 0;
          const bool chosen = by_held_row(&in, [&](auto nt, auto r) {
            threads = nt;
            pieces = r;
          });
          ++checks;
          held += chosen;
          if (chosen != (threads != 0)) return 3;
          if (chosen && rows * threads >= int64_t(1) << 32) {
            std::printf("%ld rows of %ld, type %ld: %ld threads a row\n", (long)rows, (long)vocab, (long)dt, (long)threads);
            return 4;
          }
          const int64_t piece = dt == 0 ? 4 : 8;
          if (chosen && threads * pieces < vocab / piece) return 5;
          // a batch of ordinary size whose rows fit takes it
          if (!chosen && rows >= kWantGroups && rows <= 1 << 21 && vocab / piece <= 1024 * 16) return 6;
        }
  std::printf("ok %ld %ld\n", checks, held);
  return 0;
}
