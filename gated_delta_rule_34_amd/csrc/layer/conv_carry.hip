// conv_carry.hip -- causal depthwise conv1d + SiLU with a carried window, on gfx950: prompts
// that continue from the rows before them, and one token per sequence.
//
//   z[t] = bias + sum_{j < K} w[ch][j] ext[t + j],  y[t] = z[t] sigma(z[t])
//
// with ext the K - 1 carried rows followed by the sequence's rows. What a continuation needs is
// the last K - 1 rows of ext, copied as they are. Pure streaming: each row is read and written
// once (2 ch values per row), bound by HBM; the window lives in registers. Measured (bf16, K = 4):
// 21488 rows x 10240 in 8 sequences 195 us, 4.5 TB/s (a large copy reaches 5.2); one token of 256
// sequences 17.2 us with nothing in the caches, 11 us per call in a loop; float32: 9393 rows x 10240 198 us, 3.9 TB/s.
// A wave covers 512 channels whatever their number: channels that are no multiple of 512 leave lanes of the last
// wave idle (of 16 channels, all but two).
#include "vec8.h"

namespace gdn {

// Rows [lo, hi) of sequence l, clamped into [0, rows] (a malformed table never leads outside).
__device__ __forceinline__ void carry_clamp(const ConvCarryArgs& a, int l, int64_t& lo, int64_t& hi) {
  if (!a.cu) {
    lo = (int64_t)l * a.T;
    hi = lo + a.T;
    return;
  }
  int64_t x = a.cu[l], y = a.cu[l + 1];
  x = x < 0 ? 0 : (x > a.rows ? a.rows : x);
  y = y < x ? x : (y > a.rows ? a.rows : y);
  lo = x;
  hi = y;
}

// The sequence of row t and its rows [lo, hi), by a whole wave: every step probes 64 offsets at
// once (one step up to 64 sequences, two up to 4096). A row of no sequence (behind the last one, or
// in front of cu[0] in a malformed table) gets one that does not hold it.
__device__ __forceinline__ int carry_seq(const ConvCarryArgs& a, int64_t t, int64_t& lo, int64_t& hi) {
  int l = 0;
  if (!a.cu) {
    l = (int)(t / a.T);
  } else {
    for (int n = a.N; n > 1;) {  // the largest of the n sequences from l on with cu[.] <= t
      const int stride = (n + 63) / 64, i = lane_id() * stride;
      const uint64_t m = __ballot(i < n && a.cu[l + i] <= t);
      const int at = (m ? 63 - __builtin_clzll(m) : 0) * stride;
      l += at;
      n = n - at < stride ? n - at : stride;
    }
  }
  carry_clamp(a, l, lo, hi);
  return l;
}

// Each thread owns 8 adjacent channels and RUN consecutive rows, the next PF of them in flight.
// Blocks past the runs copy one sequence's last rows each.
template <typename TI, int K, int RUN, int PF>
__global__ __launch_bounds__(64) void k_conv_prompt(ConvCarryArgs a) {
  // channel blocks run fastest, so that workgroups in flight read whole neighbouring rows
  const int yb = (a.ch / 8 + (int)blockDim.x - 1) / (int)blockDim.x, bx = (int)blockIdx.x / yb;
  int c0 = (((int)blockIdx.x - bx * yb) * (int)blockDim.x + (int)threadIdx.x) * 8;
  const bool on = c0 < a.ch;  // (idle lanes stay for the search of the sequence)
  c0 = on ? c0 : 0;
  const TI* x = (const TI*)a.x + c0;
  const TI* first = a.first ? (const TI*)a.first + c0 : nullptr;
  const int64_t runs = (a.rows + RUN - 1) / RUN;
  int64_t lo, hi;
  // Row s of sequence n's ext relative to the sequence (s < 0: carried rows).
  auto carried = [&](int n, int64_t s) -> F8 {
    return first ? ld8<TI>(first + ((int64_t)n * (K - 1) + (K - 1) + s) * a.ch) : zero8();
  };
  if (bx >= runs) {
    const int n = (int)(bx - runs);
    carry_clamp(a, n, lo, hi);
    TI* last = (TI*)a.last + c0;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int64_t s = hi - lo - (K - 1) + j;
      const F8 v = s >= 0 ? ld8<TI>(x + (lo + s) * a.x_rs) : carried(n, s);
      if (on) st8<TI>(last + ((int64_t)n * (K - 1) + j) * a.ch, v);
    }
    return;
  }
  const int64_t t0 = (int64_t)bx * RUN;
  const int64_t t1 = t0 + RUN < a.rows ? t0 + RUN : a.rows;
  TI* y = (TI*)a.y + c0;
  Raw8<TI> buf[PF];
#pragma unroll
  for (int u = 0; u < PF; ++u)
    if (t0 + u < t1) buf[u] = ldraw8<true, TI>(x + (t0 + u) * a.x_rs);
  // the rows in front of the run, used if they belong to its sequence
  F8 win[K > 1 ? K - 1 : 1];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) win[j] = t0 - (K - 1) + j >= 0 ? ld8<TI>(x + (t0 - (K - 1) + j) * a.x_rs) : zero8();
  float w[K][8], bias[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][i] = a.w[(int64_t)(c0 + i) * K + j];
    bias[i] = a.bias ? a.bias[c0 + i] : 0.f;
  }
  auto enter = [&](int64_t t) {  // places of row t's window in front of its sequence: carried rows, or none
    const int n = carry_seq(a, t, lo, hi);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int64_t s = t - lo - (K - 1) + j;
      if (t < lo || t >= hi) win[j] = zero8();
      else if (s < 0) win[j] = carried(n, s);
    }
  };
  enter(t0);
  for (int64_t base = t0; base < t1; base += PF) {
#pragma unroll
    for (int u = 0; u < PF; ++u) {
      const int64_t t = base + u;
      if (t >= t1) break;
      const F8 xt = cvt8<TI>(buf[u]);
      if (t + PF < t1) buf[u] = ldraw8<true, TI>(x + (t + PF) * a.x_rs);
      if (t >= hi && t > t0) enter(t);
      F8 out;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float z = bias[i] + w[K - 1][i] * xt.v[i];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) z += w[j][i] * win[j].v[i];
        out.v[i] = z * sigmoidf<TI>(z);
      }
      if (on && t >= lo && t < hi) st8nt<TI>(y + t * a.y_rs, out);  // rows of no sequence stay as they were
#pragma unroll
      for (int j = 0; j + 1 < K - 1; ++j) win[j] = win[j + 1];
      if constexpr (K > 1) win[K - 2] = xt;
    }
  }
}

// One token: grid (rows / R, channel blocks). The window is read, moved on by one row and written.
// A thread takes R rows of its channels: their loads are in flight together, and the weights, which
// its lanes read 32 K bytes apart, are read once for all of them.
template <typename TI, int K, int R> __global__ __launch_bounds__(64) void k_conv_decode(ConvCarryArgs a) {
  const int c0 = (int)(blockIdx.y * blockDim.x + threadIdx.x) * 8;
  if (c0 >= a.ch) return;
  Raw8<TI> xr[R], sr[R][K > 1 ? K - 1 : 1];
  int slot[R];
#pragma unroll
  for (int u = 0; u < R; ++u) {
    const int n = (int)blockIdx.x * R + u;
    slot[u] = n >= a.N ? -1 : a.idx ? a.idx[n] : n;
    if (slot[u] >= a.n_slots) slot[u] = -1;
    if (slot[u] < 0) continue;  // the row is skipped
    xr[u] = ldraw8<false, TI>((const TI*)a.x + (int64_t)n * a.x_rs + c0);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) sr[u][j] = ldraw8<false, TI>((const TI*)a.state + ((int64_t)slot[u] * (K - 1) + j) * a.ch + c0);
  }
  float w[K][8], bias[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][i] = a.w[(int64_t)(c0 + i) * K + j];
    bias[i] = a.bias ? a.bias[c0 + i] : 0.f;
  }
#pragma unroll
  for (int u = 0; u < R; ++u) {
    if (slot[u] < 0) continue;
    const F8 xt = cvt8<TI>(xr[u]);
    F8 out;
#pragma unroll
    for (int i = 0; i < 8; ++i) out.v[i] = bias[i] + w[K - 1][i] * xt.v[i];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const F8 s = cvt8<TI>(sr[u][j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) out.v[i] += w[j][i] * s.v[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) out.v[i] *= sigmoidf<TI>(out.v[i]);
    TI* st = (TI*)a.state + (int64_t)slot[u] * (K - 1) * a.ch + c0;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) straw8<TI>(st + (int64_t)j * a.ch, j + 1 < K - 1 ? sr[u][j + 1 < K - 1 ? j + 1 : j] : xr[u]);
    st8<TI>((TI*)a.y + (int64_t)((int)blockIdx.x * R + u) * a.y_rs + c0, out);
  }
}

// One-wave workgroups (512 channels): a token step of 256 rows x 10240 channels spreads over 1280 of
// them and takes 17.5 us, over 320 of four waves 20.
constexpr int kConvWave = 64;
static int conv_blocks(int ch) { return (ch / 8 + kConvWave - 1) / kConvWave; }

template <typename TI, int K, int RUN, int PF> static void prompt_run(const ConvCarryArgs& a, hipStream_t s) {
  const int64_t blocks = (a.rows + RUN - 1) / RUN + (a.last && K > 1 ? a.N : 0);
  if (blocks == 0) return;
  const unsigned grid = (unsigned)(blocks * conv_blocks(a.ch));
  traced("k_conv_prompt", s, [&] { k_conv_prompt<TI, K, RUN, PF><<<grid, kConvWave, 0, s>>>(a); });
}

// Long runs amortise a run's weights, window and search; short ones leave no compute unit idle.
// Measured (bf16, K = 4): 21488 x 10240 in 64-row runs 197 us, in 16-row ones 243; 2048 x 10240 45
// and 28 us; 512 x 2048 38 and 14, in 8-row ones 11 us.
template <typename TI, int K> static hipError_t prompt_k(const ConvCarryArgs& a, hipStream_t s) {
  const int64_t long_runs = (a.rows + 63) / 64 * conv_blocks(a.ch);
  if (long_runs >= 2048) prompt_run<TI, K, 64, 2>(a, s);
  else if (long_runs >= 256) prompt_run<TI, K, 16, 4>(a, s);
  else prompt_run<TI, K, 8, 8>(a, s);
  return hipGetLastError();
}

// Rows per thread of a decode step: four once that leaves every compute unit a workgroup.
template <typename TI, int K> static hipError_t decode_k(const ConvCarryArgs& a, hipStream_t s) {
  const int yb = conv_blocks(a.ch);
  if ((int64_t)a.N * yb >= 4 * 256) {
    const dim3 grid((unsigned)((a.N + 3) / 4), (unsigned)yb);
    traced("k_conv_decode", s, [&] { k_conv_decode<TI, K, 4><<<grid, kConvWave, 0, s>>>(a); });
  } else {
    const dim3 grid((unsigned)a.N, (unsigned)yb);
    traced("k_conv_decode", s, [&] { k_conv_decode<TI, K, 1><<<grid, kConvWave, 0, s>>>(a); });
  }
  return hipGetLastError();
}

template <typename TI> static hipError_t conv_t(const ConvCarryArgs& a, bool decode, hipStream_t s) {
  switch (a.K) {
    case 1: return decode ? decode_k<TI, 1>(a, s) : prompt_k<TI, 1>(a, s);
    case 2: return decode ? decode_k<TI, 2>(a, s) : prompt_k<TI, 2>(a, s);
    case 3: return decode ? decode_k<TI, 3>(a, s) : prompt_k<TI, 3>(a, s);
    case 4: return decode ? decode_k<TI, 4>(a, s) : prompt_k<TI, 4>(a, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_conv_prompt(const ConvCarryArgs& a, int dtype, hipStream_t s) {
  return dtype == 0 ? conv_t<float>(a, false, s) : conv_t<__bf16>(a, false, s);
}

hipError_t launch_conv_decode(const ConvCarryArgs& a, int dtype, hipStream_t s) {
  if (a.N == 0) return hipSuccess;
  return dtype == 0 ? conv_t<float>(a, true, s) : conv_t<__bf16>(a, true, s);
}

}  // namespace gdn
