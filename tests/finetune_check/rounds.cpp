// The cases of cases.cpp with so few workgroups a launch, and so small a size
// from which buffers go past the caches, that a few dozen rows take every loop
// of the kernels around: layer norm's rounds over rows (with groups that have no
// row in the last one), and the forms of the losses and the clipping for large
// buffers.
//
//   rounds [small]     small: what ThreadSanitizer runs within a minute
#define FINETUNE_NORM_GROUPS 1     // 8 workgroups of 256 threads forward, 1 or 2 backward
#define FINETUNE_CACHE_BYTES 8192  // of a call's large buffers

#define main cases_main
#include "cases.cpp"
#undef main

int main(int argc, char** argv) {
  const bool small = argc > 1 && std::string(argv[1]) == "small";
  for (int dt = 0; dt < 3; ++dt) {
    if (small && dt == 2) continue;
    layer_norm_case(560, 5, dt, 1, 1, false);  // 8 threads a row, 32 rows a workgroup: 18 groups of rows, the last half empty
    layer_norm_case(17, 1999, dt, 1, 1, false);  // 128: two waves a row, two rows a workgroup, the last pair without its second
    if (small && dt != 1) continue;
    layer_norm_case(300, 128, dt, 0, 0, true);  // ... whole pieces
    layer_norm_case(150, 250, dt, 3, 1, true);  // 16
    layer_norm_case(75, 500, dt, 0, 0, false);  // 32
    layer_norm_case(37, 1000, dt, 1, 3, true);  // a wave
    layer_norm_case(19, 2000, dt, 0, 0, true);  // 128
    loss_case(2, 40, 150, dt, 7, 3, true, true);  // a wave a row, past the caches
    layer_norm_case(11, 4093, dt, 1, 1, true);   // 256
    layer_norm_case(9, 8190, dt, 0, 0, true);    // 512
    layer_norm_case(5, 16383, dt, 1, 1, false);  // 1024: sums in LDS, no row loaded ahead in fp32
    loss_case(2, 5, 4300, dt, 1, 5, true, false);  // rows held by 256 threads
    if (small) continue;
    layer_norm_case(5, 16384, dt, 0, 0, true);
    layer_norm_case(40, 16400, dt, 3, 1, true);  // the kernels of any length, three ranges of rows
    loss_case(2, 36, 2100, dt, 1, 1, false, false);
    loss_case(2, 4, 20011, dt, 1, 1, true, false);
  }
  clip_case({5, 1, 0, 17}, 1, 1, false, 0.5);
  clip_case({90000, 3, 40961}, 3, 5, false, 1.0);
  clip_case({33, 81921, 7}, 2, 2, true, 1.0);
  std::printf("ok %ld %ld\n", cases, emu::launches);
  return 0;
}
