// Low-rank adapters of many requests at once, beside a projection that all
// rows share:
//
//   out[t, :] = y[t, :] + scale_i B_i (A_i x_t),   i the adapter of row t
//
// with A_i [rank, k] and B_i [n, rank] in bf16.  Both products run over the
// runs of a plan, so that a tile of rows meets one adapter.
//
// Two launches.  "down" makes u = A x: a block takes a tile of places and a
// part of k, its waves take pieces of 128 of that part, all of the rank at
// once; their sums are added in LDS in a fixed order and stored in binary32,
// one buffer for each part.  "up" adds the parts in their order and makes
// out = y + scale B u: each wave owns 128 columns of a tile of rows.  u enters
// the second product as a sum of two bf16 values (16 bits of mantissa), which
// is as good as binary32 beside the bf16 B and costs nothing that shows: the
// second product is bound by reading y and writing out.  The MFMA's rows are
// columns of out in an order that leaves each lane eight neighbours (tile
// pair a, lane quarter q: columns 32 a + 8 q ..), so that y and out move in
// 16-byte pieces, 64 bytes of a row at a time.
//
// Rows without an adapter come last in the plan: they are copied, or left
// alone where out is y.
#include "moe.hpp"
#include "decode_ops.hpp"

namespace qlin {
namespace {

__device__ __forceinline__ floatx4 mfma(bf16x8_t a, bf16x8_t b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ bf16x8_t load8(const uint16_t* p) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  return as_bf16x8(u32x4{v.x, v.y, v.z, v.w});
}

__device__ __forceinline__ int row_of(const RowPlan& p, int place) {
  return int(min(uint32_t(p.order[place]), uint32_t(p.rows - 1)));
}

// MT tiles of 16 places, RT tiles of 16 of the rank (the last may be half).
template <int MT, int RT>
__global__ __launch_bounds__(512) void lora_down_kernel(LoraArgs A, int parts) {
  constexpr int WAVES = 8;
  __shared__ floatx4 red[WAVES][RT * MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = blockIdx.x % parts;
  const RowTile tile = find_tile(A.plan, 16 * MT, blockIdx.x / parts);
  if (tile.group < 0 || tile.group == A.plan.groups) return;
  const int q = lane >> 4, r = lane & 15;
  const int G = A.k / 128;
  const int g0 = int(int64_t(G) * part / parts), g1 = int(int64_t(G) * (part + 1) / parts);

  const uint16_t* xr[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xr[m] = static_cast<const uint16_t*>(A.x) +
            row_of(A.plan, tile.first + min(16 * m + r, tile.count - 1)) * A.x_stride + 8 * q;
  const uint16_t* ar[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
    ar[i] = static_cast<const uint16_t*>(A.a) +
            (int64_t(tile.group) * A.rank + min(16 * i + r, A.rank - 1)) * A.k + 8 * q;

  floatx4 acc[RT][MT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = floatx4{0.f, 0.f, 0.f, 0.f};
  for (int g = g0 + wave; g < g1; g += WAVES) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8_t xf[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) xf[m] = load8(xr[m] + g * 128 + 32 * s);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const bf16x8_t af = load8(ar[i] + g * 128 + 32 * s);
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[i][m] = mfma(af, xf[m], acc[i][m]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) red[wave][i * MT + m][lane] = acc[i][m];
  __syncthreads();
  for (int t = threadIdx.x; t < RT * MT * 64; t += 512) {
    const int i = t / 64 / MT, m = t / 64 % MT, ln = t % 64;
    floatx4 sum = red[0][t / 64][ln];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += red[w][t / 64][ln];
    const int place = 16 * m + (ln & 15), j = 16 * i + 4 * (ln >> 4);
    if (place < tile.count && j < A.rank)   // the rank is a multiple of 8
      *reinterpret_cast<floatx4*>(A.part + (int64_t(part) * A.plan.rows + tile.first + place) * A.rank + j) = sum;
  }
}

// KT pieces of 32 of the rank.
template <int MT, int KT, bool kBF16>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs A, int parts, int col_blocks) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col0 = (int(blockIdx.x % col_blocks) * 4 + wave) * 128;
  const RowTile tile = find_tile(A.plan, 16 * MT, blockIdx.x / col_blocks);
  if (tile.group < 0 || col0 >= A.n) return;
  const bool bare = tile.group == A.plan.groups;
  if (bare && A.out == A.y) return;
  const int q = lane >> 4, r = lane & 15;

  // u of the tile's places, in two bf16 values each
  bf16x8_t hi[MT][KT], lo[MT][KT];
  int row[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int place = tile.first + min(16 * m + r, tile.count - 1);
    row[m] = row_of(A.plan, place);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const int j = 32 * kt + 8 * q;
      floatx4 u[2] = {floatx4{0.f, 0.f, 0.f, 0.f}, floatx4{0.f, 0.f, 0.f, 0.f}};
      if (!bare && j < A.rank) {
        const float* p = A.part + int64_t(place) * A.rank + j;
        for (int s = 0; s < parts; ++s, p += int64_t(A.plan.rows) * A.rank) {
          u[0] += *reinterpret_cast<const floatx4*>(p);
          u[1] += *reinterpret_cast<const floatx4*>(p + 4);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = u[e >> 2][e & 3];
        const __bf16 h = static_cast<__bf16>(v);
        hi[m][kt][e] = h;
        lo[m][kt][e] = static_cast<__bf16>(v - static_cast<float>(h));
      }
    }
  }
  const float scale = bare ? 0.f : A.scale ? A.scale[tile.group] : 1.0f;
  const uint16_t* b = static_cast<const uint16_t*>(A.b) + int64_t(bare ? 0 : tile.group) * A.n * A.rank;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int col = col0 + 32 * a + 8 * q;   // this lane's eight columns
    floatx4 acc[2][MT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[i][m] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (!bare) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = min(col0 + 32 * a + 8 * (r >> 2) + 4 * i + (r & 3), A.n - 1);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          const int j = 32 * kt + 8 * q;
          bf16x8_t bf = as_bf16x8(u32x4{0u, 0u, 0u, 0u});
          if (j < A.rank) bf = load8(b + int64_t(n) * A.rank + j);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            acc[i][m] = mfma(bf, hi[m][kt], acc[i][m]);
            acc[i][m] = mfma(bf, lo[m][kt], acc[i][m]);
          }
        }
      }
    }
    if (col >= A.n) continue;   // n is a multiple of 16
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (16 * m + r >= tile.count) continue;
      if constexpr (kBF16) {
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(A.y) +
                                                        row[m] * A.y_stride + col);
        const uint32_t d[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = pack_bf16x2(
              fmaf(scale, acc[e >> 1][m][2 * (e & 1)], __uint_as_float(d[e] << 16)),
              fmaf(scale, acc[e >> 1][m][2 * (e & 1) + 1], __uint_as_float(d[e] & 0xFFFF0000u)));
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.out) + row[m] * A.out_stride + col) =
            bare ? v : make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        const floatx4* from = reinterpret_cast<const floatx4*>(static_cast<const float*>(A.y) + row[m] * A.y_stride + col);
        floatx4* to = reinterpret_cast<floatx4*>(static_cast<float*>(A.out) + row[m] * A.out_stride + col);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const floatx4 v = from[i];
          floatx4 o;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = fmaf(scale, acc[i][m][e], v[e]);
          to[i] = bare ? v : o;
        }
      }
    }
  }
}

// The height of a tile: 64 places (32 beside a rank over 64, whose sums would
// not fit in LDS) where adapters have that many rows on average, else 16.
int tall_of(int64_t rows, int64_t groups, int rank) {
  return rows < 48 * groups ? 16 : rank > 64 ? 32 : 64;
}

// Parts of k: as many as fill the chip once, at least 512 of k each.
int parts_of(int64_t rows, int64_t groups, int rank, int64_t k) {
  const int cus = device_cu_count();
  const int64_t tiles = most_tiles(rows, groups, tall_of(rows, groups, rank));
  int64_t parts = (cus > 0 ? cus : 256) / (tiles > 0 ? tiles : 1);
  if (parts > k / 512) parts = k / 512;
  return parts < 1 ? 1 : int(parts);
}

template <int MT, int RT>
hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  const int parts = parts_of(a.plan.rows, a.plan.groups, a.rank, a.k);
  const int64_t tiles = most_tiles(a.plan.rows, a.plan.groups, 16 * MT);
  lora_down_kernel<MT, RT><<<unsigned(tiles * parts), 512, 0, s>>>(a, parts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int cols = (a.n + 511) / 512;
  constexpr int KT = (RT + 1) / 2;
  if (a.y_dtype == 1)
    lora_up_kernel<MT, KT, true><<<unsigned(tiles * cols), 256, 0, s>>>(a, parts, cols);
  else
    lora_up_kernel<MT, KT, false><<<unsigned(tiles * cols), 256, 0, s>>>(a, parts, cols);
  return hipGetLastError();
}

}  // namespace

size_t lora_ws_bytes(int64_t rows, int64_t groups, int rank, int64_t k) {
  return size_t(parts_of(rows, groups, rank, k)) * size_t(rows) * size_t(rank) * sizeof(float);
}

hipError_t launch_lora_add(const LoraArgs& a, hipStream_t s) {
  const int tall = tall_of(a.plan.rows, a.plan.groups, a.rank);
  if (a.rank <= 16) return tall == 16 ? launch_lora<1, 1>(a, s) : launch_lora<4, 1>(a, s);
  if (a.rank <= 32) return tall == 16 ? launch_lora<1, 2>(a, s) : launch_lora<4, 2>(a, s);
  if (a.rank <= 64) return tall == 16 ? launch_lora<1, 4>(a, s) : launch_lora<4, 4>(a, s);
  return tall == 16 ? launch_lora<1, 8>(a, s) : launch_lora<2, 8>(a, s);
}

}  // namespace qlin
