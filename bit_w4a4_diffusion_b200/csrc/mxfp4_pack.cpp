// Host-side (untimed) MXFP4 weight preparation and the scale-layout helpers.
// The rounding works on the fp32 fields, with no code in common with the
// device quantizer; both follow the OCP MX definition and give equal bytes.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <system_error>
#include <thread>
#include <vector>

#include "svdq.h"

namespace svdq {
int record_error(int status, const char* fmt, ...);
}

namespace {

using svdq::record_error;

// Magnitude (already divided by the block's scale) -> 3-bit E2M1 code.
// Midpoints go to the even code.
uint8_t e2m1_magnitude(float a) {
  static const float kMid[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.0f};
  int c = 0;
  for (int i = 0; i < 7; ++i)
    if (a > kMid[i] || (a == kMid[i] && (i & 1))) c = i + 1;
  return (uint8_t)c;
}

size_t tile_offset(long long row, int group, int K) {
  const size_t chunks = ((size_t)K + 127) / 128;
  return ((size_t)(row >> 7) * chunks + (group >> 2)) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4 + (group & 3);
}

// f(i) for every i in [0, n) on the host's threads.  Threads that cannot be
// had leave their share to this one.
template <class F>
void parallel_rows(long long n, F&& f) {
  unsigned nt = std::max(1u, std::min(16u, std::thread::hardware_concurrency()));
  if (n < 64) nt = 1;
  auto share = [&](unsigned t) {
    for (long long i = t; i < n; i += nt) f(i);
  };
  std::vector<std::thread> th;
  unsigned t = 1;
  try {
    th.reserve(nt);
    for (; t < nt; ++t) th.emplace_back(share, t);
  } catch (const std::exception&) {
  }
  share(0);
  for (; t < nt; ++t) share(t);
  for (auto& x : th) x.join();
}

bool shape_ok(int matrices, int N, int K) { return matrices > 0 && N > 0 && K > 0 && K % 32 == 0; }

}  // namespace

extern "C" {

int mxfp4_pack_weights(int matrices, int N, int K, const uint16_t* W, uint8_t* codes, uint8_t* scales) {
  if (!shape_ok(matrices, N, K))
    return record_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "matrices=%d N=%d K=%d: positive, K a multiple of 32",
                        matrices, N, K);
  if (!W || !codes || !scales) return record_error(SVDQ_ERR_INVALID_ARG, "null pointer argument");
  const size_t per = (size_t)mxfp4_scale_bytes(N, K);
  std::memset(scales, 0, per * matrices);
  parallel_rows((long long)matrices * N, [&](long long row) {
    const uint16_t* w = W + (size_t)row * K;
    uint8_t* c = codes + (size_t)row * (K / 2);
    uint8_t* sc = scales + per * (size_t)(row / N);
    for (int g = 0; g < K / 32; ++g) {
      uint16_t top = 0;
      for (int i = 0; i < 32; ++i) top = std::max<uint16_t>(top, w[32 * g + i] & 0x7FFF);
      const int e = top >> 7;   // bf16 exponent field
      const int b = e == 255 ? 255 : std::max(e - 2, 0);
      sc[tile_offset(row % N, g, K)] = (uint8_t)b;
      for (int i = 0; i < 32; i += 2) {
        uint8_t pair = 0;
        for (int h = 0; h < 2 && b != 255; ++h) {
          const uint32_t u = (uint32_t)w[32 * g + i + h] << 16;
          float v;
          std::memcpy(&v, &u, 4);
          const uint8_t code = e2m1_magnitude(std::ldexp(std::fabs(v), 127 - b)) | (std::signbit(v) ? 8 : 0);
          pair |= (uint8_t)(code << (4 * h));
        }
        c[16 * g + i / 2] = pair;
      }
    }
  });
  return SVDQ_OK;
}

int mxfp4_scales_to_rowmajor(int matrices, int rows, int K, const uint8_t* tiled, uint8_t* rowmajor) {
  if (!shape_ok(matrices, rows, K))
    return record_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "matrices=%d rows=%d K=%d: positive, K a multiple of 32",
                        matrices, rows, K);
  if (!tiled || !rowmajor) return record_error(SVDQ_ERR_INVALID_ARG, "null pointer argument");
  const size_t per = (size_t)mxfp4_scale_bytes(rows, K);
  for (long long r = 0; r < (long long)matrices * rows; ++r)
    for (int g = 0; g < K / 32; ++g)
      rowmajor[(size_t)r * (K / 32) + g] = tiled[per * (size_t)(r / rows) + tile_offset(r % rows, g, K)];
  return SVDQ_OK;
}

int mxfp4_scales_from_rowmajor(int matrices, int rows, int K, const uint8_t* rowmajor, uint8_t* tiled) {
  if (!shape_ok(matrices, rows, K))
    return record_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "matrices=%d rows=%d K=%d: positive, K a multiple of 32",
                        matrices, rows, K);
  if (!tiled || !rowmajor) return record_error(SVDQ_ERR_INVALID_ARG, "null pointer argument");
  const size_t per = (size_t)mxfp4_scale_bytes(rows, K);
  std::memset(tiled, 0, per * matrices);
  for (long long r = 0; r < (long long)matrices * rows; ++r)
    for (int g = 0; g < K / 32; ++g)
      tiled[per * (size_t)(r / rows) + tile_offset(r % rows, g, K)] = rowmajor[(size_t)r * (K / 32) + g];
  return SVDQ_OK;
}

}  // extern "C"
