// api.hip -- the C ABI of libswizzled_gemm.so: argument validation, the
// variant plan (tile shape, grid, raster) and the launch on the caller's
// stream.  Every check runs before any HIP call, so each error path is
// reachable on a machine without a GPU.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>

#include "../../include/swizzled_gemm.h"
#include "i8_params.h"
#include "launch.h"
#include "lds_layout.h"
#include "moe.h"
#include "xent_plan.h"

namespace {

thread_local std::string g_last_error;
// The clock trace of this thread's launches (gemm_clock_trace); off by default.
thread_local sg::ClockTrace g_clk{nullptr, 0};

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

int ok() {
  g_last_error.clear();
  return SG_OK;
}

int elem_bytes(int dt) {
  switch (dt) {
    case SG_F16:
    case SG_BF16:
      return 2;
    case SG_F32:
      return 4;
    case SG_E4M3:
    case SG_E8M0:
      return 1;
    default:
      return 0;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool is_out_dtype(int dt) { return dt == SG_F32 || dt == SG_BF16 || dt == SG_F16; }

constexpr int64_t kMaxExtent = (int64_t)1 << 31;  // buffer offsets are 32-bit
using sg::kCUs;
constexpr int kGroupM = 8;

// Largest byte extent one workgroup addresses through a buffer resource
// (ld = the operand's leading dimension in elements).
int64_t panel_extent(int major, int64_t rows, int64_t K, int64_t ld, int64_t tile_rows,
                     int eb) {
  if (K == 0) return 0;
  return major == SG_K_MAJOR ? ((rows < tile_rows ? rows : tile_rows) - 1) * ld * eb + K * eb
                             : (K - 1) * ld * eb + rows * eb;
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Grouped GEMM and MXFP8: 256x256 tiles when they fill the CUs, or when
// 128x128 tiles would need two or more rounds of the CUs and 256-row panels
// stay within 32-bit buffer offsets (`fits256`); else 128x128 tiles.  Their
// 128x128 kernels trail the 256x256 ping-pongs further than the dense one
// does (MI355X, TFLOP/s 256 vs 128 tiles: MXFP8 2560^3 1176 vs 1014, 3072^3
// 1738 vs 803, 3840^3 2263 vs 1316; grouped bf16 4 x 512 x 4096 x 4096 1055
// vs 1015, 4 x 768 x 4096 x 4096 1345 vs 913), but not one round of them
// (MXFP8 2048^3 755 vs 796).
sg::TileShape pick_tile(int64_t tiles256, int64_t tiles128, bool fits256) {
  if (tiles256 >= kCUs) return sg::kTile256;
  if (fits256 && cdiv(tiles128, kCUs) >= 2) return sg::kTile256;
  return sg::kTile128;
}

int64_t tile_rows(sg::TileShape t) { return t == sg::kTile256 ? 256 : t == sg::kTile128 ? 128 : 64; }

int hip_fail(hipError_t e, const char* what) {
  return fail(SG_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// Which kernels dense_run launches.
enum DenseMode { kLibrary, kAblation256, kAblation128, kAblationIO };

// gemm_run, gemm_strided_run, gemm_layout_run and gemm_layout128_run:
// validation, plan and launch.  kLibrary runs the library's kernels; the
// ablation modes run the layout `swz` (16, 8, 0, or padded on 128x128
// tiles) on the 256x256 or 128x128 kernel whatever the problem size.
// Leading dimensions are in elements.
int dense_run(const char* who, DenseMode mode, int swz, int64_t M, int64_t N, int64_t K,
              float alpha,
              const void* A, int64_t lda, int a_major, const void* B, int64_t ldb,
              int b_major, int ab_dtype, float beta, const void* C, int64_t ldc, int c_dtype,
              void* D, int64_t ldd, int d_dtype, void* stream) {
  if (M < 0 || N < 0 || K < 0)
    return fail(SG_ERR_SHAPE, "%s: negative size M=%lld N=%lld K=%lld", who,
                (long long)M, (long long)N, (long long)K);
  if (ab_dtype != SG_F16 && ab_dtype != SG_BF16)
    return fail(SG_ERR_DTYPE, "%s: ab_dtype %d is not SG_F16/SG_BF16", who, ab_dtype);
  if (!is_out_dtype(d_dtype))
    return fail(SG_ERR_DTYPE, "%s: d_dtype %d is not SG_F32/SG_BF16/SG_F16", who, d_dtype);
  if (C && !is_out_dtype(c_dtype))
    return fail(SG_ERR_DTYPE, "%s: c_dtype %d is not SG_F32/SG_BF16/SG_F16", who, c_dtype);
  if (C && C == D && (c_dtype != d_dtype || ldc != ldd))
    return fail(SG_ERR_DTYPE, "%s: in-place C == D needs c_dtype == d_dtype and ldc == ldd",
                who);
  if ((a_major != SG_K_MAJOR && a_major != SG_MN_MAJOR) ||
      (b_major != SG_K_MAJOR && b_major != SG_MN_MAJOR))
    return fail(SG_ERR_MAJOR, "%s: majorness must be SG_K_MAJOR or SG_MN_MAJOR", who);
  if (lda < (a_major == SG_K_MAJOR ? K : M) || ldb < (b_major == SG_K_MAJOR ? K : N) ||
      ldd < N || (C && ldc < N))
    return fail(SG_ERR_SHAPE,
                "%s: a leading dimension is below its minimum (lda %lld, ldb %lld, ldc %lld, "
                "ldd %lld)", who, (long long)lda, (long long)ldb, (long long)ldc,
                (long long)ldd);
  if (N % 4)
    return fail(SG_ERR_SHAPE, "%s: N=%lld is not a multiple of 4 (D is written 4 columns at "
                              "a time)", who, (long long)N);
  if (M == 0 || N == 0) return ok();
  if (!D) return fail(SG_ERR_NULL, "%s: D is NULL", who);
  // alpha == 0: A and B are not read; beta == 0: C is not read.
  if (alpha == 0.0f) K = 0;
  if (beta == 0.0f) C = nullptr;
  if (K > 0 && (!A || !B)) return fail(SG_ERR_NULL, "%s: A or B is NULL", who);
  const int eb = 2, db = elem_bytes(d_dtype), cb = C ? elem_bytes(c_dtype) : 0;
  if ((K > 0 && (!aligned16(A) || !aligned16(B))) || !aligned16(D) || (C && !aligned16(C)))
    return fail(SG_ERR_ALIGN, "%s: every pointer must be 16-byte aligned", who);
  if ((K > 0 && ((lda * eb) % 16 || (ldb * eb) % 16)) || (ldd * db) % 16 ||
      (C && (ldc * cb) % 16))
    return fail(SG_ERR_ALIGN,
                "%s: row pitches must be multiples of 16 bytes (A %lld, B %lld, D %lld bytes)",
                who, (long long)(lda * eb), (long long)(ldb * eb), (long long)(ldd * db));
  // The loaders move whole 16-byte chunks of a K-major row: with K % 8 != 0
  // the elements past K in the last chunk would come from the row padding.
  // (Packed rows cannot get here: their pitch 2K is then not a multiple of 16.)
  if (K > 0 && K % 8 && (a_major == SG_K_MAJOR || b_major == SG_K_MAJOR))
    return fail(SG_ERR_SHAPE, "%s: K=%lld is not a multiple of 8 with a K-major operand",
                who, (long long)K);
  const bool fits256 = panel_extent(a_major, M, K, lda, 256, eb) < kMaxExtent &&
                       panel_extent(b_major, N, K, ldb, 256, eb) < kMaxExtent;
  const sg::TileShape tile = mode == kAblation256 || mode == kAblationIO ? sg::kTile256
                            : mode == kAblation128 ? sg::kTile128
                                                   : sg::pick_dense_tile(
                                                         M, N,
                                                         (a_major == SG_K_MAJOR &&
                                                          b_major == SG_K_MAJOR) ||
                                                             (K % 64 == 0 && K >= 128),
                                                         fits256);
  const int64_t T = tile_rows(tile);
  if (panel_extent(a_major, M, K, lda, T, eb) >= kMaxExtent ||
      panel_extent(b_major, N, K, ldb, T, eb) >= kMaxExtent ||
      lda * eb >= kMaxExtent || ldb * eb >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "%s: an operand panel spans 2^31 bytes or more", who);
  const int64_t tiles_m = cdiv(M, T), tiles_n = cdiv(N, T);
  if (tiles_m * tiles_n >= kMaxExtent || tiles_m * tiles_n > 0x7fffffffLL)
    return fail(SG_ERR_SHAPE, "%s: too many tiles", who);

  sg::DenseParams p;
  p.A = A;
  p.B = B;
  p.C = C;
  p.D = D;
  p.M = M;
  p.N = N;
  p.K = K;
  p.lda = lda;
  p.ldb = ldb;
  p.ldc = C ? ldc : 0;
  p.ldd = ldd;
  p.alpha = alpha;
  p.beta = C ? beta : 0.0f;
  p.c_dtype = C ? c_dtype : SG_NONE;
  p.d_dtype = d_dtype;
  p.tiles_m = (int)tiles_m;
  p.tiles_n = (int)tiles_n;
  p.group_m = kGroupM;
  p.clk = g_clk;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = mode == kAblationIO    ? sg::launch_layout_io(swz & 0xff, swz >> 8, p, s)
                       : mode == kAblation256 ? sg::launch_layout(swz, p, s)
                       : mode == kAblation128 ? sg::launch_layout128(swz, p, s)
                                              : sg::launch_dense(tile, ab_dtype == SG_BF16,
                                                                 a_major == SG_MN_MAJOR,
                                                                 b_major == SG_MN_MAJOR, p, s);
  if (e != hipSuccess) return hip_fail(e, who);
  return ok();
}

}  // namespace

namespace sg {
const char*& last_kernel() {
  thread_local const char* name = "";
  return name;
}
}  // namespace sg

extern "C" {

const char* gemm_last_kernel(void) { return sg::last_kernel(); }

const char* gemm_last_error(void) { return g_last_error.c_str(); }

const char* gemm_version(void) {
  return "swizzled_gemm 0.3 (gfx950; 16-bit MFMA 16x16x32 and 32x32x16, MXFP8/MXFP6/MXFP4 "
         "scaled MFMA 32x32x64; LDS XOR swizzle over 256-byte bank lines)";
}

int gemm_run(int64_t M, int64_t N, int64_t K, const void* A, int a_major,
             const void* B, int b_major, int ab_dtype, const void* C, int c_dtype,
             void* D, int d_dtype, void* stream) {
  return dense_run("gemm_run", kLibrary, 0, M, N, K, 1.0f, A, a_major == SG_K_MAJOR ? K : M, a_major,
                   B, b_major == SG_K_MAJOR ? K : N, b_major, ab_dtype, 1.0f, C, N, c_dtype,
                   D, N, d_dtype, stream);
}

int gemm_strided_run(int64_t M, int64_t N, int64_t K, float alpha, const void* A,
                     int64_t lda, int a_major, const void* B, int64_t ldb, int b_major,
                     int ab_dtype, float beta, const void* C, int64_t ldc, int c_dtype,
                     void* D, int64_t ldd, int d_dtype, void* stream) {
  return dense_run("gemm_strided_run", kLibrary, 0, M, N, K, alpha, A, lda, a_major, B, ldb, b_major,
                   ab_dtype, beta, C, ldc, c_dtype, D, ldd, d_dtype, stream);
}

int gemm_layout_run(int swz_units, int64_t M, int64_t N, int64_t K, const void* A,
                    const void* B, const void* C, int c_dtype, void* D, int d_dtype,
                    void* stream) {
  if (swz_units != 0 && swz_units != 8 && swz_units != 16)
    return fail(SG_ERR_SHAPE, "gemm_layout_run: swz_units %d is not 0, 8 or 16", swz_units);
  return dense_run("gemm_layout_run", kAblation256, swz_units, M, N, K, 1.0f, A, K,
                   SG_K_MAJOR, B, K, SG_K_MAJOR, SG_BF16, 1.0f, C, N, c_dtype, D, N, d_dtype,
                   stream);
}

int gemm_layout_io_run(int operand_swz, int output_swz, int64_t M, int64_t N, int64_t K,
                       const void* A, const void* B, const void* C, int c_dtype, void* D,
                       int d_dtype, void* stream) {
  if (operand_swz != 0 && operand_swz != 16)
    return fail(SG_ERR_SHAPE, "gemm_layout_io_run: operand_swz %d is not 0 or 16", operand_swz);
  if (output_swz != 0 && output_swz != 1)
    return fail(SG_ERR_SHAPE, "gemm_layout_io_run: output_swz %d is not 0 or 1", output_swz);
  if (d_dtype != SG_BF16 && d_dtype != SG_F16)
    return fail(SG_ERR_DTYPE, "gemm_layout_io_run: d_dtype %d is not 16-bit (a 16-bit D is "
                              "what the epilogue stages in LDS)", d_dtype);
  if (C && c_dtype != SG_BF16 && c_dtype != SG_F16)
    return fail(SG_ERR_DTYPE, "gemm_layout_io_run: c_dtype %d is not 16-bit", c_dtype);
  return dense_run("gemm_layout_io_run", kAblationIO, operand_swz | (output_swz << 8), M, N, K,
                   1.0f, A, K, SG_K_MAJOR, B, K, SG_K_MAJOR, SG_BF16, 1.0f, C, N, c_dtype, D,
                   N, d_dtype, stream);
}

int gemm_layout128_run(int layout, int64_t M, int64_t N, int64_t K, const void* A,
                       const void* B, const void* C, int c_dtype, void* D, int d_dtype,
                       void* stream) {
  if (layout != 0 && layout != 8 && layout != 16 && layout != SG_LAYOUT_PAD16)
    return fail(SG_ERR_SHAPE, "gemm_layout128_run: layout %d is not 0, 8, 16 or "
                "SG_LAYOUT_PAD16", layout);
  return dense_run("gemm_layout128_run", kAblation128,
                   layout == SG_LAYOUT_PAD16 ? sg::kSwzPad : layout, M, N, K, 1.0f, A, K,
                   SG_K_MAJOR, B, K, SG_K_MAJOR, SG_BF16, 1.0f, C, N, c_dtype, D, N, d_dtype,
                   stream);
}

int grouped_gemm_run(int G, const int64_t* m_offsets, int64_t N, int64_t K,
                     const void* A, int a_major, const void* B, int b_major,
                     int ab_dtype, void* D, int d_dtype, void* stream) {
  if (G < 1 || G > SG_MAX_GROUPS)
    return fail(SG_ERR_GROUPS, "grouped_gemm_run: G=%d outside [1, %d]", G, SG_MAX_GROUPS);
  if (!m_offsets) return fail(SG_ERR_NULL, "grouped_gemm_run: m_offsets is NULL");
  if (m_offsets[0] != 0)
    return fail(SG_ERR_GROUPS, "grouped_gemm_run: m_offsets[0] must be 0");
  for (int g = 0; g < G; ++g)
    if (m_offsets[g + 1] < m_offsets[g])
      return fail(SG_ERR_GROUPS, "grouped_gemm_run: m_offsets decrease at group %d", g);
  if (N < 0 || K < 0)
    return fail(SG_ERR_SHAPE, "grouped_gemm_run: negative size N=%lld K=%lld",
                (long long)N, (long long)K);
  if (ab_dtype != SG_F16 && ab_dtype != SG_BF16)
    return fail(SG_ERR_DTYPE, "grouped_gemm_run: ab_dtype %d is not SG_F16/SG_BF16", ab_dtype);
  if (!is_out_dtype(d_dtype))
    return fail(SG_ERR_DTYPE, "grouped_gemm_run: d_dtype %d unsupported", d_dtype);
  if (a_major != SG_K_MAJOR || b_major != SG_K_MAJOR)
    return fail(SG_ERR_MAJOR, "grouped_gemm_run: A and B must be SG_K_MAJOR");
  const int64_t total = m_offsets[G];
  if (total == 0 || N == 0) return ok();
  if (!D) return fail(SG_ERR_NULL, "grouped_gemm_run: D is NULL");
  if (K > 0 && (!A || !B)) return fail(SG_ERR_NULL, "grouped_gemm_run: A or B is NULL");
  const int eb = 2, db = elem_bytes(d_dtype);
  if ((K > 0 && (!aligned16(A) || !aligned16(B))) || !aligned16(D))
    return fail(SG_ERR_ALIGN, "grouped_gemm_run: every pointer must be 16-byte aligned");
  if ((K * eb) % 16 || (N * db) % 16)
    return fail(SG_ERR_ALIGN, "grouped_gemm_run: row pitches must be multiples of 16 bytes");
  int64_t tiles256 = 0, tiles128 = 0;
  for (int g = 0; g < G; ++g) {
    tiles256 += cdiv(m_offsets[g + 1] - m_offsets[g], 256);
    tiles128 += cdiv(m_offsets[g + 1] - m_offsets[g], 128);
  }
  tiles256 *= cdiv(N, 256);
  tiles128 *= cdiv(N, 128);
  const sg::TileShape tile = pick_tile(tiles256, tiles128, 256 * K * eb < kMaxExtent);
  const int64_t T = tile == sg::kTile256 ? 256 : 128;
  if (T * K * eb >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "grouped_gemm_run: an operand panel spans 2^31 bytes or more");
  sg::GroupedParams p;
  p.A = A;
  p.B = B;
  p.D = D;
  p.N = N;
  p.K = K;
  p.d_dtype = d_dtype;
  p.G = G;
  p.tiles_n = (int)cdiv(N, T);
  p.group_m = kGroupM;
  p.clk = g_clk;
  int64_t acc = 0;
  for (int g = 0; g <= G; ++g) {
    p.m_off[g] = m_offsets[g];
    p.tile_start[g] = (int32_t)acc;
    if (g < G) acc += cdiv(m_offsets[g + 1] - m_offsets[g], T) * p.tiles_n;
    if (acc > 0x7fffffffLL) return fail(SG_ERR_SHAPE, "grouped_gemm_run: too many tiles");
  }
  for (int g = G + 1; g <= SG_MAX_GROUPS; ++g) {
    p.m_off[g] = m_offsets[G];
    p.tile_start[g] = (int32_t)acc;
  }
  if (acc == 0) return ok();
  hipError_t e = sg::launch_grouped(tile, ab_dtype == SG_BF16, sg::kSwzDefault, p,
                                    (int)acc, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "grouped_gemm_run launch");
  return ok();
}

namespace {

// The shared checks and launch of the block-scaled GEMMs: fmt SG_E4M3,
// SG_E2M1, SG_E2M3 or SG_E3M2; scales in layout sf_layout (SG_SF_ROWS: 4-byte
// aligned; SG_SF_BLOCKS: 16-byte aligned).
int mx_run(const char* who, int fmt, int sf_layout, int64_t M, int64_t N, int64_t K,
           const void* A, const void* SFA, const void* B, const void* SFB, void* D,
           int d_dtype, void* stream) {
  const bool fp4 = fmt == SG_E2M1, fp6 = fmt == SG_E2M3 || fmt == SG_E3M2;
  if (fmt != SG_E4M3 && !fp4 && !fp6)
    return fail(SG_ERR_DTYPE, "%s: fmt %d is not SG_E4M3/SG_E2M1/SG_E2M3/SG_E3M2", who, fmt);
  if (sf_layout != SG_SF_ROWS && sf_layout != SG_SF_BLOCKS)
    return fail(SG_ERR_SHAPE, "%s: sf_layout %d is not SG_SF_ROWS/SG_SF_BLOCKS", who, sf_layout);
  if (M < 0 || N < 0 || K < 0) return fail(SG_ERR_SHAPE, "%s: negative size", who);
  const int64_t kmul = fp4 ? 256 : 128;
  if (K % kmul)
    return fail(SG_ERR_SHAPE, "%s: K=%lld is not a multiple of %lld", who, (long long)K,
                (long long)kmul);
  if (d_dtype != SG_F32 && d_dtype != SG_BF16)
    return fail(SG_ERR_DTYPE, "%s: d_dtype %d is not SG_F32/SG_BF16", who, d_dtype);
  if (M == 0 || N == 0) return ok();
  if (!D) return fail(SG_ERR_NULL, "%s: D is NULL", who);
  if (K > 0 && (!A || !B || !SFA || !SFB))
    return fail(SG_ERR_NULL, "%s: A, B, SFA or SFB is NULL", who);
  const int db = elem_bytes(d_dtype);
  const uintptr_t sf_mask = sf_layout == SG_SF_BLOCKS ? 15u : 3u;
  if ((K > 0 && (!aligned16(A) || !aligned16(B))) || !aligned16(D) ||
      (K > 0 && ((reinterpret_cast<uintptr_t>(SFA) | reinterpret_cast<uintptr_t>(SFB)) & sf_mask)))
    return fail(SG_ERR_ALIGN, "%s: A, B, D must be 16-byte aligned, SFA and SFB %d-byte aligned",
                who, sf_layout == SG_SF_BLOCKS ? 16 : 4);
  if ((N * db) % 16)
    return fail(SG_ERR_ALIGN, "%s: D row pitch must be a multiple of 16 bytes", who);
  // MXFP8 takes 128x128 tiles for small problems; the others 256x256.
  const int64_t row_bytes = fp4 ? K / 2 : fp6 ? K / 4 * 3 : K;
  const bool fits256 = 256 * row_bytes < kMaxExtent &&
                       (sf_layout != SG_SF_BLOCKS || 4 * cdiv(K, 512) * 1024 < kMaxExtent);
  const sg::TileShape tile =
      fmt == SG_E4M3 ? pick_tile(cdiv(M, 256) * cdiv(N, 256), cdiv(M, 128) * cdiv(N, 128), fits256)
                     : sg::kTile256;
  const int64_t T = tile == sg::kTile256 ? 256 : 128;
  // a tile's panel (plus, for fp6, the 8 bytes its shifted rows may read beyond it)
  if (T * row_bytes + (fp6 ? 8 : 0) >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "%s: an operand panel spans 2^31 bytes or more", who);
  if (sf_layout == SG_SF_BLOCKS && cdiv(T, 64) * cdiv(K, 512) * 1024 >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "%s: a tile's scales span 2^31 bytes or more", who);
  const int64_t tiles_m = cdiv(M, T), tiles_n = cdiv(N, T);
  if (tiles_m * tiles_n > 0x7fffffffLL) return fail(SG_ERR_SHAPE, "%s: too many tiles", who);
  sg::MxParams p;
  p.A = A;
  p.SFA = SFA;
  p.B = B;
  p.SFB = SFB;
  p.D = D;
  p.M = M;
  p.N = N;
  p.K = K;
  p.d_dtype = d_dtype;
  p.sf_layout = sf_layout;
  p.tiles_m = (int)tiles_m;
  p.tiles_n = (int)tiles_n;
  p.group_m = kGroupM;
  p.clk = g_clk;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = fp4   ? sg::launch_mxfp4(p, s)
                       : fp6 ? sg::launch_mxfp6(fmt == SG_E3M2, p, s)
                             : sg::launch_mx(tile, p, s);
  if (e != hipSuccess) return fail(SG_ERR_HIP, "%s launch: %s", who, hipGetErrorString(e));
  return ok();
}

}  // namespace

int mxfp4_gemm_run(int64_t M, int64_t N, int64_t K, const void* A, const void* SFA,
                   const void* B, const void* SFB, void* D, int d_dtype, void* stream) {
  return mx_run("mxfp4_gemm_run", SG_E2M1, SG_SF_ROWS, M, N, K, A, SFA, B, SFB, D, d_dtype,
                stream);
}

int mxfp6_gemm_run(int fmt, int64_t M, int64_t N, int64_t K, const void* A, const void* SFA,
                   const void* B, const void* SFB, void* D, int d_dtype, void* stream) {
  if (fmt != SG_E2M3 && fmt != SG_E3M2)
    return fail(SG_ERR_DTYPE, "mxfp6_gemm_run: fmt %d is not SG_E2M3/SG_E3M2", fmt);
  return mx_run("mxfp6_gemm_run", fmt, SG_SF_ROWS, M, N, K, A, SFA, B, SFB, D, d_dtype, stream);
}

int mx_gemm_run(int64_t M, int64_t N, int64_t K, const void* A, const void* SFA,
                const void* B, const void* SFB, void* D, int d_dtype, void* stream) {
  return mx_run("mx_gemm_run", SG_E4M3, SG_SF_ROWS, M, N, K, A, SFA, B, SFB, D, d_dtype,
                stream);
}

int mx_gemm_blocks_run(int fmt, int64_t M, int64_t N, int64_t K, const void* A,
                       const void* SFA, const void* B, const void* SFB, void* D, int d_dtype,
                       void* stream) {
  return mx_run("mx_gemm_blocks_run", fmt, SG_SF_BLOCKS, M, N, K, A, SFA, B, SFB, D, d_dtype,
                stream);
}

int64_t mx_scales_blocks_bytes(int64_t rows, int64_t K) {
  if (rows < 0 || K < 0 || K % 32)
    return fail(SG_ERR_SHAPE, "mx_scales_blocks_bytes: rows=%lld K=%lld (K a multiple of 32)",
                (long long)rows, (long long)K);
  return cdiv(rows, 64) * cdiv(K, 512) * 1024;
}

int mx_scales_to_blocks(const void* SF, int64_t rows, int64_t K, void* out, void* stream) {
  if (rows < 0 || K < 0 || K % 128)
    return fail(SG_ERR_SHAPE, "mx_scales_to_blocks: rows=%lld K=%lld (K a multiple of 128)",
                (long long)rows, (long long)K);
  if (rows == 0 || K == 0) return ok();
  if (!SF || !out) return fail(SG_ERR_NULL, "mx_scales_to_blocks: SF or out is NULL");
  if ((reinterpret_cast<uintptr_t>(SF) & 3u) || !aligned16(out))
    return fail(SG_ERR_ALIGN, "mx_scales_to_blocks: SF must be 4-byte, out 16-byte aligned");
  if (cdiv(rows, 64) > 0x7fffffffLL || cdiv(cdiv(K, 512), 16) > 65535)
    return fail(SG_ERR_SHAPE, "mx_scales_to_blocks: too many rows or K blocks");
  hipError_t e = sg::launch_sf_blocks(SF, rows, K, out, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "mx_scales_to_blocks launch");
  return ok();
}

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int64_t kI8MaxK = 131056;  // 2^14 * K < 2^31, K a multiple of 16
// A launch has fewer than 2^32 threads along x, 512 a tile.  (A grid over x and
// y would take more; 2^23 tiles are 2^29 columns of one row, or 2^37 outputs.)
constexpr int64_t kI8MaxTiles = (int64_t{1} << 23) - 1;

struct I8Shape {
  int64_t rows, cols;
};
I8Shape i8_shape(sg::I8Tile t) {
  switch (t) {
    case sg::kI8Stream16x16: return {16, 16};
    case sg::kI8Stream16x32: return {16, 32};
    case sg::kI8Stream16x64: return {16, 64};
    case sg::kI8Stream32x16: return {32, 16};
    case sg::kI8Stream32x32:
    case sg::kI8Stream32x32x2: return {32, 32};
    case sg::kI8Stream64x32: return {64, 32};
    case sg::kI8Mid64x64: return {64, 64};
    case sg::kI8Mid64x128: return {64, 128};
    case sg::kI8Mid128x128: return {128, 128};
    default: return {256, 256};
  }
}

// The streaming kernel for up to 64 rows (16 when grouped) and `cols` columns
// of B in all.  Narrow tiles while 16 columns a workgroup are no more
// workgroups than CUs, then 32 (MI355X, us, 16 / 32 / 64 columns: 1 x 4096 x
// 4096 5.5 / 6.0 / 7.0; 1 x 8192 x 8192 15.4 / 15.0 / 16.6); 64 where there
// are many workgroups of few stages each.  How many changes with the columns
// (us, 32 / 64, by K):
//                          1024       2048       2560       3328       4096
//   1 x 33024           11.4 10.0  19.1 19.5  20.2 22.8  25.0 29.2  33.2 37.8
//   1 x 65536           20.9 17.7  30.3 27.7  32.8 32.1  42.2 40.7  53.5 56.2
//   16 x 131072         40.0 30.7  57.5 54.2  69.6 64.3  84.3 79.6  94.9 104
//   64 experts of 2048  48.0 35.4  66.9 56.2  70.3 66.9  86.4 83.1  103  106
//   128 experts of 1024 48.6 34.9  66.9 56.3  70.9 67.0  87.1 83.3  103  106
// Up to K = 2048, 64 columns cost at most 5% and gain up to 27%; beyond, they
// gain at most 8% where there are many and lose 13 to 17% where there are few.
// 17 to 32 rows: five stages for one workgroup a CU, two stages for more (32 x
// 8192 x 8192 16.5 / 20.0, 32 x 28672 x 8192 55 / 49).
sg::I8Tile pick_i8_stream(int64_t M, int64_t cols, int64_t K) {
  const bool narrow = cols <= 16 * kCUs;
  if (M <= 16)
    return narrow ? sg::kI8Stream16x16
                  : cols > 128 * kCUs && K <= 2048 ? sg::kI8Stream16x64 : sg::kI8Stream16x32;
  if (M <= 32)
    return narrow ? sg::kI8Stream32x16
                  : cols <= 32 * kCUs ? sg::kI8Stream32x32 : sg::kI8Stream32x32x2;
  return sg::kI8Stream64x32;
}

// The tile of a larger product: the least of a model of the time, in ns.  A
// round of workgroups costs `start` (tile lookup, first loads, epilogue) and,
// for each 128 bytes of K, `step` alone and `full` with every CU busy (the
// smaller the tile, the sooner the L2's rate limits it, about 17 TB/s in all).
// The rows are fitted to MI355X times of 64 to 4096 rows by 4096 and 8192
// columns (us, model / measured / the best other tile): 128 x 4096 x 4096
// 64x64 10.0 / 9.6 / 12.7; 333 x 4104 x 4112 64x128 16.5 / 18.0 / 21.3; 768 x
// 4096 x 4096 128x128 22.3 / 21.2 / 27.7; 2048 x 4096 x 4096 256x256 44 / 42.8
// / 47.6; 1024 x 8192 x 8192 256x256 81 / 77.8 / 83.8.
struct I8Cost {
  sg::I8Tile tile;
  double start, step, full;
};
constexpr I8Cost kI8Costs[] = {{sg::kI8Mid64x64, 2500, 140, 210},
                               {sg::kI8Mid64x128, 3500, 210, 350},
                               {sg::kI8Mid128x128, 5000, 300, 550},
                               {sg::kI8PingPong256, 6500, 950, 1300}};
sg::I8Tile pick_i8_tile(int64_t M, int64_t groups, int64_t N, int64_t K, bool fits256) {
  sg::I8Tile best = sg::kI8Mid64x64;
  double least = 0;
  for (const I8Cost& c : kI8Costs) {
    if (c.tile == sg::kI8PingPong256 && !fits256) continue;
    const I8Shape s = i8_shape(c.tile);
    // Row tiles: every group's last one is half empty on average.
    const double rows = groups == 1 ? (double)cdiv(M, s.rows)
                                    : (double)M / s.rows + 0.5 * (double)groups;
    const double wgs = (rows > (double)groups ? rows : (double)groups) * (double)cdiv(N, s.cols);
    const double rounds = (double)(int64_t)(wgs / kCUs), left = wgs / kCUs - rounds;
    const double k = (double)cdiv(K, 128);
    double ns = rounds * (c.start + k * c.full);
    if (left > 0) ns += c.start + k * (c.step + (c.full - c.step) * left);
    if (least == 0 || ns < least) {
      least = ns;
      best = c.tile;
    }
  }
  return best;
}

// Dense: streaming up to 64 rows (for 33 to 64 only while its workgroups fit
// the CUs: 64 x 8192 x 8192 19.4 us against 64x64 tiles' 25.8, 64 x 16384 x
// 2048 13.1 against 9.9).
sg::I8Tile pick_i8_dense(int64_t M, int64_t N, int64_t K, bool fits256) {
  if (M <= 32 || (M <= 64 && N <= 32 * kCUs)) return pick_i8_stream(M, N, K);
  return pick_i8_tile(M, 1, N, K, fits256);
}

// Grouped, from the groups' mean rows (the offsets are in device memory).  Up
// to 8 rows a group on average stream (64 experts of 2048 x 2048, us, 64x128
// tiles / streaming: 4 rows 60 / 47, 16 rows 60 / 68).  Beyond, each group's B
// comes from memory whatever the tile, so 256x256 tiles win as soon as they
// fill the CUs (64 experts of 2048 x 2048 with 64 rows each 64x128 / 128x128 /
// 256x256: 70 / 79 / 64 us; 256 rows 203 / 160 / 91).
sg::I8Tile pick_i8_grouped(int64_t R, int64_t G, int64_t N, int64_t K, bool fits256) {
  const int64_t groups = G < R ? G : R;
  if (cdiv(R, G) <= 8) return pick_i8_stream(1, groups * N, K);
  if (fits256 && (groups > R / 256 ? groups : R / 256) * cdiv(N, 256) >= kCUs)
    return sg::kI8PingPong256;
  return pick_i8_tile(R, groups, N, K, fits256);
}

// The shared checks and launch of the 8-bit products; G = 0: dense.
int i8_run(const char* who, int G, int64_t M, int64_t N, int64_t K, const int32_t* offsets,
           const void* A, int64_t lda, const int32_t* rows, int64_t a_rows, const float* SA,
           const void* B, int64_t ldb, const float* SB, void* D, int64_t ldd, int d_dtype,
           void* stream) {
  if (M < 0 || N < 0 || K < 0 || a_rows < 0)
    return fail(SG_ERR_SHAPE, "%s: negative size M=%lld N=%lld K=%lld", who, (long long)M,
                (long long)N, (long long)K);
  if (!is_out_dtype(d_dtype))
    return fail(SG_ERR_DTYPE, "%s: d_dtype %d is not SG_F32/SG_BF16/SG_F16", who, d_dtype);
  if (K % 16 || K > kI8MaxK)
    return fail(SG_ERR_SHAPE, "%s: K=%lld is not a multiple of 16 up to %lld", who, (long long)K,
                (long long)kI8MaxK);
  if (lda < K || ldb < K || ldd < N)
    return fail(SG_ERR_SHAPE, "%s: a leading dimension is below its minimum (lda %lld, ldb %lld, "
                              "ldd %lld)", who, (long long)lda, (long long)ldb, (long long)ldd);
  if (M >= kMaxExtent || N >= kMaxExtent || a_rows >= kMaxExtent || lda >= kMaxExtent ||
      ldb >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "%s: 2^31 rows or columns or more, or such a pitch", who);
  if (M == 0 || N == 0) return ok();
  if (!D || (G > 0 && !offsets)) return fail(SG_ERR_NULL, "%s: D or offsets is NULL", who);
  const bool no_a = rows && a_rows == 0;  // no index names a row
  if ((K > 0 && !no_a && !A) || (K > 0 && !B) || (!no_a && !SA) || !SB)
    return fail(SG_ERR_NULL, "%s: A, B, SA or SB is NULL", who);
  const int db = elem_bytes(d_dtype);
  if ((K > 0 && (!aligned16(A) || !aligned16(B))) || !aligned4(SA) || !aligned4(SB) ||
      !aligned4(offsets) || !aligned4(rows) || reinterpret_cast<uintptr_t>(D) % db)
    return fail(SG_ERR_ALIGN, "%s: A and B must be 16-byte aligned, the other pointers to their "
                              "elements", who);
  if (lda % 16 || ldb % 16)
    return fail(SG_ERR_ALIGN, "%s: the row pitches of A and B must be multiples of 16 bytes", who);
  if (rows && a_rows > 0 && (a_rows - 1) * lda + K >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "%s: gathered A spans 2^31 bytes or more", who);
  const bool fits256 = 256 * lda < kMaxExtent && 256 * ldb < kMaxExtent;
  const sg::I8Tile tile = G == 0 ? pick_i8_dense(M, N, K, fits256)
                                 : pick_i8_grouped(M, G, N, K, fits256);
  const int64_t T = i8_shape(tile).rows, tn = i8_shape(tile).cols;
  if ((T > tn ? T : tn) * (lda > ldb ? lda : ldb) >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "%s: an operand panel spans 2^31 bytes or more", who);
  const int64_t tiles_n = cdiv(N, tn);
  // Row tiles: every group may end in a partial one.
  const int64_t groups = G == 0 ? 1 : G < M ? G : M;
  const int64_t tiles_m = G == 0 ? cdiv(M, T) : (M + groups * (T - 1)) / T;
  if (tiles_m * tiles_n > kI8MaxTiles)
    return fail(SG_ERR_SHAPE, "%s: %lld tiles of %lld x %lld, at most %lld in a call", who,
                (long long)(tiles_m * tiles_n), (long long)T, (long long)tn,
                (long long)kI8MaxTiles);
  sg::I8Params p;
  p.A = A;
  p.B = B;
  p.SA = SA;
  p.SB = SB;
  p.D = D;
  p.M = M;
  p.N = N;
  p.K = K;
  p.lda = lda;
  p.ldb = ldb;
  p.ldd = ldd;
  p.d_dtype = d_dtype;
  p.vec = aligned16(D) && (ldd * db) % 16 == 0;
  p.tiles_m = (int)tiles_m;
  p.tiles_n = (int)tiles_n;
  p.group_m = kGroupM;
  p.clk = g_clk;
  p.G = G;
  p.offsets = offsets;
  p.rows = rows;
  p.a_total = (int)a_rows;
  const hipError_t e = sg::launch_i8(tile, p, (int)(tiles_m * tiles_n),
                                     static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, who);
  return ok();
}

// The checks that the cross entropy and its gradient share.
int xent_check(const char* who, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
               const void* B, int64_t ldb, int ab_dtype, const void* targets, int target_dtype) {
  if (M < 0 || N < 0 || K < 0 || M >= kMaxExtent || N >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "%s: M=%lld, N=%lld (both below 2^31), K=%lld", who, (long long)M,
                (long long)N, (long long)K);
  if (ab_dtype != SG_F16 && ab_dtype != SG_BF16)
    return fail(SG_ERR_DTYPE, "%s: ab_dtype %d is not SG_F16/SG_BF16", who, ab_dtype);
  if (target_dtype != SG_I32 && target_dtype != SG_I64)
    return fail(SG_ERR_DTYPE, "%s: target_dtype %d is not SG_I32/SG_I64", who, target_dtype);
  if (K % 8) return fail(SG_ERR_SHAPE, "%s: K=%lld is not a multiple of 8", who, (long long)K);
  if (lda < K || ldb < K || lda >= sg::kXentMaxLd || ldb >= sg::kXentMaxLd)
    return fail(SG_ERR_SHAPE, "%s: lda=%lld, ldb=%lld outside [K=%lld, 2^22)", who,
                (long long)lda, (long long)ldb, (long long)K);
  if (lda % 8 || ldb % 8)
    return fail(SG_ERR_ALIGN, "%s: the row pitches of A and B must be multiples of 16 bytes", who);
  if (M > 0 && !targets) return fail(SG_ERR_NULL, "%s: targets is NULL", who);
  if (K > 0 && ((M > 0 && !A) || (N > 0 && !B)))
    return fail(SG_ERR_NULL, "%s: A or B is NULL", who);
  if (!aligned16(A) || !aligned16(B) ||
      reinterpret_cast<uintptr_t>(targets) % (target_dtype == SG_I64 ? 8 : 4))
    return fail(SG_ERR_ALIGN, "%s: A and B must be 16-byte aligned, targets to its elements", who);
  const int64_t side = sg::tile_side(sg::xent_tile(M, N));
  if (cdiv(M, side) * cdiv(N, side) >= sg::kXentMaxTiles)
    return fail(SG_ERR_SHAPE, "%s: 2^23 or more tiles of %lld x %lld", who, (long long)side,
                (long long)side);
  return SG_OK;
}

sg::XentCall xent_call(int64_t M, int64_t N, int64_t K, float alpha, const void* A, int64_t lda,
                       const void* B, int64_t ldb, int ab_dtype, const void* targets,
                       int target_dtype, void* workspace) {
  sg::XentCall c{};
  c.M = M;
  c.N = N;
  c.K = K;
  c.alpha = alpha;
  c.A = A;
  c.lda = lda;
  c.B = B;
  c.ldb = ldb;
  c.bf16 = ab_dtype == SG_BF16;
  c.targets = targets;
  c.wide = target_dtype == SG_I64;
  c.workspace = workspace;
  return c;
}

int workspace_check(const char* who, const void* workspace, int64_t bytes, int64_t need) {
  if (bytes < need)
    return fail(SG_ERR_SHAPE, "%s: the workspace has %lld bytes, %lld are needed", who,
                (long long)bytes, (long long)need);
  if (need > 0 && !workspace) return fail(SG_ERR_NULL, "%s: workspace is NULL", who);
  if (!aligned16(workspace))
    return fail(SG_ERR_ALIGN, "%s: workspace must be 16-byte aligned", who);
  return SG_OK;
}

// Rows of a call's argument in memory, in bytes (a vector: one row).
struct Area {
  const char* name;
  const void* at;
  int64_t rows, pitch, width;
};

// Whether two areas have a byte in common.  Rows of one pitch may lie side by
// side; of two pitches only areas one behind the other are known to be apart.
bool overlap(const Area& a, const Area& b) {
  if (!a.at || !b.at || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.at), pb = reinterpret_cast<uintptr_t>(b.at);
  if (pa > pb) return overlap(b, a);
  const uintptr_t from = pb - pa;
  if (from >= (uintptr_t)(a.rows - 1) * (uintptr_t)a.pitch + (uintptr_t)a.width) return false;
  const int64_t pitch = a.rows > 1 ? a.pitch : b.pitch;
  if (a.rows > 1 && b.rows > 1 && a.pitch != b.pitch) return true;
  const int64_t column = (int64_t)(from % (uintptr_t)pitch);
  return column < a.width || column + b.width > pitch;
}

// No output (the first `outputs` areas) overlaps another area.
int overlap_check(const char* who, const Area* areas, int outputs, int all) {
  for (int i = 0; i < outputs; ++i)
    for (int k = i + 1; k < all; ++k)
      if (overlap(areas[i], areas[k]))
        return fail(SG_ERR_ALIGN, "%s: %s overlaps %s", who, areas[i].name, areas[k].name);
  return SG_OK;
}

// The checks that the forward and backward routing share.
int route_check(const char* who, int64_t T, int E, int top_k, const void* logits, int64_t ldl,
                int dtype, int score) {
  if (T < 0 || T >= kMaxExtent || E < 1 || E > SG_MAX_GROUPS || top_k < 1 || top_k > E ||
      top_k > SG_MAX_TOP_K)
    return fail(SG_ERR_SHAPE, "%s: T=%lld, E=%d (1..%d), top_k=%d (1..min(E, %d))", who,
                (long long)T, E, SG_MAX_GROUPS, top_k, SG_MAX_TOP_K);
  if (!is_out_dtype(dtype))
    return fail(SG_ERR_DTYPE, "%s: dtype %d is not SG_F32/SG_BF16/SG_F16", who, dtype);
  if (score != SG_SCORE_SOFTMAX && score != SG_SCORE_SIGMOID)
    return fail(SG_ERR_DTYPE, "%s: score %d is not SG_SCORE_SOFTMAX/SG_SCORE_SIGMOID", who, score);
  if (ldl < E) return fail(SG_ERR_SHAPE, "%s: ldl=%lld is below E=%d", who, (long long)ldl, E);
  if (T == 0) return SG_OK;
  if (!logits) return fail(SG_ERR_NULL, "%s: logits is NULL", who);
  if (reinterpret_cast<uintptr_t>(logits) % elem_bytes(dtype))
    return fail(SG_ERR_ALIGN, "%s: logits must be aligned to its elements", who);
  return SG_OK;
}

// Whether four values at any multiple of four of any row are one aligned access.
bool rows_of_four(const void* p, int64_t ld, int dtype) {
  return ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * elem_bytes(dtype)) == 0;
}

// Tokens that a workgroup of the balance loss adds up: one workgroup up to 256
// tokens, up to 128 workgroups for 8192 tokens, beyond that 256 (us in a graph, 64
// | 128 | 256 of them: 1024 x 256 fp32 7.5 | 7.5 | 7.5 and 9.1 for 16 of them,
// 4096 x 256 9.7 | 9.3 | 11.6, 16384 x 256 18.5 | 13.6 | 13.6, 16384 x 128 bf16
// 12.8 | 10.8 | 10.0, 65536 x 256 64 | 37 | 27; the more there are the longer the
// join reads).
int64_t balance_chunk(int64_t T) {
  return T <= 256 ? 256 : cdiv(cdiv(T, T <= 8192 ? 128 : 256), 16) * 16;
}

// Up to so many pairs the plan is one launch (us, one launch / two, 256
// experts: 8192 pairs 5.6 / 7.0, 16384 7.2 / 7.2, 32768 10.2 / 7.3).
constexpr int64_t kPlanAlone = 16384;

// Pairs that a workgroup of the plan sorts, a multiple of 64 for each of its 16
// waves.  Each of n workgroups reads n * E counts and places P / n pairs, and
// a pair takes as long as about eight counts: so n^2 E <= 8 P, fewer workgroups
// the more experts (256 experts, us, this / 1024 pairs a workgroup up to 256 of
// them: 131072 pairs 9.2 / 10.3, 524288 13.9 / 16.2).
int64_t plan_chunk(int64_t P, int E) {
  int64_t chunk = 1024;
  if (P <= kPlanAlone) return chunk;
  for (;; chunk *= 2) {
    const int64_t n = cdiv(P, chunk);
    if (n <= 256 && n * n * E <= 8 * P) return chunk;
  }
}

}  // namespace

int i8_gemm_run(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const float* SA,
                const void* B, int64_t ldb, const float* SB, void* D, int64_t ldd, int d_dtype,
                void* stream) {
  return i8_run("i8_gemm_run", 0, M, N, K, nullptr, A, lda, nullptr, M, SA, B, ldb, SB, D, ldd,
                d_dtype, stream);
}

int i8_grouped_gemm_run(int G, int64_t R, int64_t N, int64_t K, const int32_t* offsets,
                        const void* A, int64_t lda, int64_t a_rows, const int32_t* rows,
                        const float* SA, const void* B, const float* SB, void* D, int64_t ldd,
                        int d_dtype, void* stream) {
  const char* who = "i8_grouped_gemm_run";
  if (G < 1 || G > SG_MAX_GROUPS)
    return fail(SG_ERR_GROUPS, "%s: G=%d outside [1, %d]", who, G, SG_MAX_GROUPS);
  if (!rows && a_rows < R)
    return fail(SG_ERR_SHAPE, "%s: A has %lld rows, D %lld", who, (long long)a_rows,
                (long long)R);
  return i8_run(who, G, R, N, K, offsets, A, lda, rows, a_rows, SA, B, K, SB, D, ldd, d_dtype,
                stream);
}

int i8_quant_run(int64_t R, int64_t K, const void* X, int64_t ldx, int x_dtype, void* Q,
                 int64_t ldq, float* S, void* stream) {
  const char* who = "i8_quant_run";
  if (R < 0 || K < 0 || R >= kMaxExtent || K >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "%s: R=%lld K=%lld", who, (long long)R, (long long)K);
  if (!is_out_dtype(x_dtype))
    return fail(SG_ERR_DTYPE, "%s: x_dtype %d is not SG_F32/SG_BF16/SG_F16", who, x_dtype);
  if (ldx < K || ldq < cdiv(K, 16) * 16)
    return fail(SG_ERR_SHAPE, "%s: ldx=%lld is below K=%lld, or ldq=%lld below K rounded up to "
                              "16", who, (long long)ldx, (long long)K, (long long)ldq);
  if (R == 0) return ok();
  if ((K > 0 && (!X || !Q)) || !S) return fail(SG_ERR_NULL, "%s: X, Q or S is NULL", who);
  if (reinterpret_cast<uintptr_t>(X) % elem_bytes(x_dtype) || !aligned4(S) ||
      (K > 0 && (!aligned16(Q) || ldq % 16)))
    return fail(SG_ERR_ALIGN, "%s: Q and its row pitch must be 16-byte aligned, X and S to their "
                              "elements", who);
  hipError_t e = sg::launch_i8_quant(X, R, K, ldx, x_dtype, Q, ldq, S,
                                     static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, who);
  return ok();
}

int64_t gemm_xent_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0 || M >= kMaxExtent || N >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "gemm_xent_workspace_bytes: M=%lld N=%lld K=%lld", (long long)M,
                (long long)N, (long long)K);
  return sg::xent_workspace(M, N);
}

int64_t gemm_xent_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t ldb) {
  if (M < 0 || N < 0 || K < 0 || M >= sg::kXentMaxRows || N >= kMaxExtent || ldb < K ||
      ldb >= sg::kXentMaxLd)
    return fail(SG_ERR_SHAPE, "gemm_xent_backward_workspace_bytes: M=%lld (below 2^22), N=%lld, "
                              "K=%lld, ldb=%lld", (long long)M, (long long)N, (long long)K,
                (long long)ldb);
  return M == 0 || N == 0 || K == 0 ? 0 : sg::xent_plan(M, N, K, ldb).bytes;
}

int gemm_xent_run(int64_t M, int64_t N, int64_t K, float alpha, const void* A, int64_t lda,
                  const void* B, int64_t ldb, int ab_dtype, const void* targets, int target_dtype,
                  float* loss, float* lse, void* workspace, int64_t workspace_bytes,
                  void* stream) {
  const char* who = "gemm_xent_run";
  if (const int rc = xent_check(who, M, N, K, A, lda, B, ldb, ab_dtype, targets, target_dtype))
    return rc;
  if (M == 0) return ok();
  if (!loss || !lse) return fail(SG_ERR_NULL, "%s: loss or lse is NULL", who);
  if (!aligned4(loss) || !aligned4(lse))
    return fail(SG_ERR_ALIGN, "%s: loss and lse must be 4-byte aligned", who);
  if (const int rc = workspace_check(who, workspace, workspace_bytes,
                                     sg::xent_workspace(M, N)))
    return rc;
  const int64_t of_targets = M * (target_dtype == SG_I64 ? 8 : 4);
  const Area areas[] = {{"loss", loss, 1, 4 * M, 4 * M},
                        {"lse", lse, 1, 4 * M, 4 * M},
                        {"workspace", workspace, 1, workspace_bytes, sg::xent_workspace(M, N)},
                        {"A", A, M, 2 * lda, 2 * K},
                        {"B", B, N, 2 * ldb, 2 * K},
                        {"targets", targets, 1, of_targets, of_targets}};
  if (const int rc = overlap_check(who, areas, 3, 6)) return rc;
  sg::XentCall c = xent_call(M, N, K, alpha, A, lda, B, ldb, ab_dtype, targets, target_dtype,
                             workspace);
  c.loss = loss;
  c.lse = lse;
  const hipError_t e = sg::launch_xent(c, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, who);
  return ok();
}

int gemm_xent_backward_run(int64_t M, int64_t N, int64_t K, float alpha, const float* dloss,
                           const float* dlse, const void* A, int64_t lda, const void* B,
                           int64_t ldb, int ab_dtype, const void* targets, int target_dtype,
                           const float* lse, void* dA, int64_t ldda, void* dB, int64_t lddb,
                           void* workspace, int64_t workspace_bytes, void* stream) {
  const char* who = "gemm_xent_backward_run";
  if (const int rc = xent_check(who, M, N, K, A, lda, B, ldb, ab_dtype, targets, target_dtype))
    return rc;
  if (M >= sg::kXentMaxRows)
    return fail(SG_ERR_SHAPE, "%s: M=%lld is not below 2^22", who, (long long)M);
  if ((dA && ldda < K) || (dB && lddb < K))
    return fail(SG_ERR_SHAPE, "%s: ldda=%lld or lddb=%lld is below K=%lld", who, (long long)ldda,
                (long long)lddb, (long long)K);
  if ((dA && (!aligned16(dA) || ldda % 8)) || (dB && (!aligned16(dB) || lddb % 8)))
    return fail(SG_ERR_ALIGN, "%s: dA, dB and their row pitches must be 16-byte aligned", who);
  if (dB && M > 0 && ((M - 1) * lda + K) * 2 >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "%s: A spans 2^31 bytes or more, too many for dB in one call", who);
  if (M > 0 && N > 0 && K > 0 && (!dloss || !lse))
    return fail(SG_ERR_NULL, "%s: dloss or lse is NULL", who);
  if (!aligned4(dloss) || !aligned4(dlse) || !aligned4(lse))
    return fail(SG_ERR_ALIGN, "%s: dloss, dlse and lse must be 4-byte aligned", who);
  if (K == 0 || (!dA && !dB)) return ok();
  sg::XentPlan plan{};  // (half a microsecond: made once)
  if (M > 0 && N > 0) {
    plan = sg::xent_plan(M, N, K, ldb);
    if (!plan.fits)
      return fail(SG_ERR_SHAPE, "%s: a gradient of 2^23 or more tiles of 256 x 256", who);
  }
  if (const int rc = workspace_check(who, workspace, workspace_bytes, plan.bytes)) return rc;
  const int64_t of_targets = M * (target_dtype == SG_I64 ? 8 : 4);
  auto pitch = [&](int64_t rows, int64_t ld) {  // (of a single row: any, not looked at)
    return rows > 1 ? (int64_t)(2 * (uint64_t)ld) : 2 * K;
  };
  const Area areas[] = {{"dA", dA, M, pitch(M, ldda), 2 * K},
                        {"dB", dB, N, pitch(N, lddb), 2 * K},
                        {"workspace", workspace, 1, plan.bytes, plan.bytes},
                        {"A", A, M, 2 * lda, 2 * K},
                        {"B", B, N, 2 * ldb, 2 * K},
                        {"targets", targets, 1, of_targets, of_targets},
                        {"dloss", dloss, 1, 4 * M, 4 * M},
                        {"dlse", dlse, 1, 4 * M, 4 * M},
                        {"lse", lse, 1, 4 * M, 4 * M}};
  if (const int rc = overlap_check(who, areas, 3, 9)) return rc;
  sg::XentCall c = xent_call(M, N, K, alpha, A, lda, B, ldb, ab_dtype, targets, target_dtype,
                             workspace);
  c.lse = const_cast<float*>(lse);
  c.dloss = dloss;
  c.dlse = dlse;
  c.dA = dA;
  c.ldda = ldda;
  c.dB = dB;
  c.lddb = lddb;
  const hipError_t e = sg::launch_xent_backward(c, plan, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, who);
  return ok();
}

int moe_route_run(int64_t T, int E, int top_k, const void* logits, int64_t ldl, int dtype,
                  const float* bias, int score, int n_groups, int top_groups, int group_score,
                  int renorm, float scale, float* weights, int32_t* ids, void* stream) {
  const char* who = "moe_route_run";
  if (const int rc = route_check(who, T, E, top_k, logits, ldl, dtype, score)) return rc;
  if (n_groups < 1 || n_groups > SG_MAX_ROUTE_GROUPS || E % n_groups || top_groups < 1 ||
      top_groups > n_groups)
    return fail(SG_ERR_GROUPS, "%s: n_groups=%d (1..%d, dividing E=%d), top_groups=%d", who,
                n_groups, SG_MAX_ROUTE_GROUPS, E, top_groups);
  if (group_score != SG_GROUP_MAX && group_score != SG_GROUP_TOP2)
    return fail(SG_ERR_GROUPS, "%s: group_score %d is not SG_GROUP_MAX/SG_GROUP_TOP2", who,
                group_score);
  if (top_k > top_groups * (E / n_groups))
    return fail(SG_ERR_GROUPS, "%s: top_k=%d is more than the %d experts of %d groups", who, top_k,
                top_groups * (E / n_groups), top_groups);
  if (T == 0) return ok();
  if (!weights || !ids) return fail(SG_ERR_NULL, "%s: weights or ids is NULL", who);
  if (!aligned4(weights) || !aligned4(ids) || !aligned4(bias))
    return fail(SG_ERR_ALIGN, "%s: weights, ids and bias must be 4-byte aligned", who);
  sg::RouteParams p{};
  p.T = T;
  p.E = E;
  p.top_k = top_k;
  p.logits = logits;
  p.ldl = ldl;
  p.bias = bias;
  p.score = score;
  p.n_groups = top_groups == n_groups ? 1 : n_groups;  // every group kept: no choice
  p.top_groups = top_groups;
  p.group_score = group_score;
  p.renorm = renorm;
  p.scale = scale;
  p.by_score = bias || (p.n_groups > 1 && group_score == SG_GROUP_TOP2);
  p.vec = rows_of_four(logits, ldl, dtype);
  p.weights = weights;
  p.ids = ids;
  hipError_t e = sg::launch_moe_route(dtype, p, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, who);
  return ok();
}

int moe_route_backward_run(int64_t T, int E, int top_k, const float* dweights, const void* logits,
                           int64_t ldl, int dtype, const int32_t* ids, int score, int renorm,
                           float scale, void* dlogits, int64_t lddl, void* stream) {
  const char* who = "moe_route_backward_run";
  if (const int rc = route_check(who, T, E, top_k, logits, ldl, dtype, score)) return rc;
  if (lddl < E) return fail(SG_ERR_SHAPE, "%s: lddl=%lld is below E=%d", who, (long long)lddl, E);
  if (T == 0) return ok();
  if (!dweights || !ids || !dlogits)
    return fail(SG_ERR_NULL, "%s: dweights, ids or dlogits is NULL", who);
  if (!aligned4(dweights) || !aligned4(ids) ||
      reinterpret_cast<uintptr_t>(dlogits) % elem_bytes(dtype))
    return fail(SG_ERR_ALIGN, "%s: every pointer must be aligned to its elements", who);
  sg::RouteParams p{};
  p.T = T;
  p.E = E;
  p.top_k = top_k;
  p.logits = logits;
  p.ldl = ldl;
  p.score = score;
  p.renorm = renorm;
  p.scale = scale;
  p.ids = const_cast<int32_t*>(ids);
  p.dweights = dweights;
  p.dlogits = dlogits;
  p.lddl = lddl;
  p.vec = rows_of_four(logits, ldl, dtype);
  p.vec_d = rows_of_four(dlogits, lddl, dtype);
  hipError_t e = sg::launch_moe_route_backward(dtype, p, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, who);
  return ok();
}

int64_t moe_balance_workspace_bytes(int64_t T, int E) {
  if (T < 0 || T >= kMaxExtent || E < 1 || E > SG_MAX_GROUPS)
    return fail(SG_ERR_SHAPE, "moe_balance_workspace_bytes: T=%lld E=%d", (long long)T, E);
  const int64_t parts = cdiv(T, balance_chunk(T));
  return parts <= 1 ? 0 : parts * ((E + 2) & ~1) * 8;
}

int moe_balance_run(int64_t T, int E, int top_k, const void* logits, int64_t ldl, int dtype,
                    const int32_t* ids, int score, float* loss, int32_t* counts,
                    int32_t* tokens, void* workspace, int64_t workspace_bytes, void* stream) {
  const char* who = "moe_balance_run";
  if (const int rc = route_check(who, T, E, top_k, logits, ldl, dtype, score)) return rc;
  if (T * top_k >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "%s: T * top_k = %lld is not below 2^31", who,
                (long long)(T * top_k));
  if (!loss || !counts || !tokens || (T > 0 && !ids))
    return fail(SG_ERR_NULL, "%s: ids, loss, counts or tokens is NULL", who);
  if (!aligned4(ids) || !aligned4(loss) || !aligned4(counts) || !aligned4(tokens))
    return fail(SG_ERR_ALIGN, "%s: ids, loss, counts and tokens must be 4-byte aligned", who);
  if (const int rc = workspace_check(who, workspace, workspace_bytes,
                                     moe_balance_workspace_bytes(T, E)))
    return rc;
  sg::BalanceParams p{};
  p.T = T;
  p.E = E;
  p.top_k = top_k;
  p.logits = logits;
  p.ldl = ldl;
  p.score = score;
  p.vec = rows_of_four(logits, ldl, dtype);
  p.chunk = balance_chunk(T);
  p.ids = ids;
  p.loss = loss;
  p.counts = counts;
  p.tokens = tokens;
  p.part = workspace;
  p.parts = T > 0 ? (int)cdiv(T, p.chunk) : 1;
  const hipError_t e = sg::launch_moe_balance(dtype, p, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, who);
  return ok();
}

int moe_balance_backward_run(int64_t T, int E, const float* dloss, const void* logits,
                             int64_t ldl, int dtype, const int32_t* counts,
                             const int32_t* tokens, int score, void* dlogits, int64_t lddl,
                             void* stream) {
  const char* who = "moe_balance_backward_run";
  if (const int rc = route_check(who, T, E, 1, logits, ldl, dtype, score)) return rc;
  if (lddl < E) return fail(SG_ERR_SHAPE, "%s: lddl=%lld is below E=%d", who, (long long)lddl, E);
  if (T == 0) return ok();
  if (!dloss || !counts || !tokens || !dlogits)
    return fail(SG_ERR_NULL, "%s: dloss, counts, tokens or dlogits is NULL", who);
  if (!aligned4(dloss) || !aligned4(counts) || !aligned4(tokens) ||
      reinterpret_cast<uintptr_t>(dlogits) % elem_bytes(dtype))
    return fail(SG_ERR_ALIGN, "%s: every pointer must be aligned to its elements", who);
  sg::BalanceParams p{};
  p.T = T;
  p.E = E;
  p.logits = logits;
  p.ldl = ldl;
  p.score = score;
  p.vec = rows_of_four(logits, ldl, dtype);
  p.counts = const_cast<int32_t*>(counts);
  p.tokens = const_cast<int32_t*>(tokens);
  p.dloss = dloss;
  p.dlogits = dlogits;
  p.lddl = lddl;
  p.vec_d = rows_of_four(dlogits, lddl, dtype);
  const hipError_t e =
      sg::launch_moe_balance_backward(dtype, p, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, who);
  return ok();
}

int64_t moe_plan_workspace_bytes(int64_t P, int E) {
  if (P < 0 || P >= kMaxExtent || E < 1 || E > SG_MAX_GROUPS)
    return fail(SG_ERR_SHAPE, "moe_plan_workspace_bytes: P=%lld E=%d", (long long)P, E);
  return P <= kPlanAlone ? 0 : cdiv(P, plan_chunk(P, E)) * E * 4;
}

int moe_plan_run(int64_t T, int E, int top_k, const int32_t* ids, int32_t* offsets, int32_t* rows,
                 int32_t* slots, void* workspace, int64_t workspace_bytes, void* stream) {
  const char* who = "moe_plan_run";
  if (T < 0 || T >= kMaxExtent || E < 1 || E > SG_MAX_GROUPS || top_k < 1 ||
      top_k > SG_MAX_GROUPS || T * top_k >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "%s: T=%lld, E=%d (1..%d), top_k=%d (1..%d), T * top_k below 2^31",
                who, (long long)T, E, SG_MAX_GROUPS, top_k, SG_MAX_GROUPS);
  const int64_t P = T * top_k;
  if (!offsets || (P > 0 && (!ids || !rows || !slots)))
    return fail(SG_ERR_NULL, "%s: ids, offsets, rows or slots is NULL", who);
  if (!aligned4(ids) || !aligned4(offsets) || !aligned4(rows) || !aligned4(slots) ||
      !aligned4(workspace))
    return fail(SG_ERR_ALIGN, "%s: every pointer must be 4-byte aligned", who);
  const int64_t need = moe_plan_workspace_bytes(P, E);
  if (workspace_bytes < need)
    return fail(SG_ERR_SHAPE, "%s: the workspace has %lld bytes, %lld are needed", who,
                (long long)workspace_bytes, (long long)need);
  if (need > 0 && !workspace) return fail(SG_ERR_NULL, "%s: workspace is NULL", who);
  sg::PlanParams p;
  p.P = P;
  p.E = E;
  p.top_k = top_k;
  p.chunk = plan_chunk(P, E);
  p.ids = ids;
  p.offsets = offsets;
  p.rows = rows;
  p.slots = slots;
  p.counts = need > 0 ? static_cast<int32_t*>(workspace) : nullptr;
  p.div_shift = top_k > 1 ? 32 - __builtin_clz(top_k - 1) : 0;
  p.div_mul = (uint32_t)(((1ull << 32) * ((1ull << p.div_shift) - top_k)) / top_k + 1);
  hipError_t e = sg::launch_moe_plan(p, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, who);
  return ok();
}

int gemm_clock_trace(void* buf, int64_t slots, int* wall_khz) {
  if (slots < 0) return fail(SG_ERR_SHAPE, "gemm_clock_trace: slots=%lld < 0", (long long)slots);
  if (buf && (reinterpret_cast<uintptr_t>(buf) & 7u))
    return fail(SG_ERR_ALIGN, "gemm_clock_trace: buf must be 8-byte aligned");
  if (wall_khz) {
    int dev = 0, khz = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&khz, hipDeviceAttributeWallClockRate, dev);
    if (e != hipSuccess) return hip_fail(e, "gemm_clock_trace: wall clock rate");
    *wall_khz = khz;
  }
  g_clk.buf = static_cast<uint64_t*>(buf);
  g_clk.slots = buf ? slots : 0;
  return ok();
}

int gemm_clock_probe(int64_t iters, void* out, void* stream) {
  if (!out) return fail(SG_ERR_NULL, "gemm_clock_probe: out is NULL");
  if (reinterpret_cast<uintptr_t>(out) & 7u)
    return fail(SG_ERR_ALIGN, "gemm_clock_probe: out must be 8-byte aligned");
  if (iters < 1 || iters > (int64_t{1} << 24))
    return fail(SG_ERR_SHAPE, "gemm_clock_probe: iters=%lld outside [1, 2^24]",
                (long long)iters);
  hipError_t e = sg::launch_clock_probe(iters, out, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "gemm_clock_probe launch");
  return ok();
}

int gemm_clock_probe_waves(void) { return sg::clock_probe_waves(); }

int gemm_lds_layout(int rows, int row_bytes, int32_t* out) {
  if (!out) return fail(SG_ERR_NULL, "gemm_lds_layout: out is NULL");
  if (rows <= 0 || rows % 8 || (row_bytes != 64 && row_bytes != 128 && row_bytes != 256))
    return fail(SG_ERR_SHAPE, "gemm_lds_layout: rows must be a positive multiple of 8 "
                              "and row_bytes 64, 128 or 256");
  const int chunks = row_bytes / 16;
  for (int r = 0; r < rows; ++r)
    for (int c = 0; c < chunks; ++c)
      out[r * chunks + c] = (int32_t)sg::lds_offset_rt(row_bytes, sg::kSwzDefault, r, c);
  return ok();
}

int gemm_lds_layout_mxfp6(int rows, int unshifted, int32_t* out) {
  if (!out) return fail(SG_ERR_NULL, "gemm_lds_layout_mxfp6: out is NULL");
  if (rows <= 0 || rows % 32 || unshifted < 0 || unshifted > 32)
    return fail(SG_ERR_SHAPE, "gemm_lds_layout_mxfp6: rows must be a positive multiple of 32 "
                              "and unshifted in [0, 32]");
  for (int r = 0; r < rows; ++r)
    for (int q = 0; q < 12; ++q)
      out[r * 12 + q] = (int32_t)sg::mxfp6_lds_offset(r, 8u * q, (uint32_t)unshifted);
  return ok();
}

int gemm_lds_layout_cblock(int32_t* out) {
  if (!out) return fail(SG_ERR_NULL, "gemm_lds_layout_cblock: out is NULL");
  for (int w = 0; w < 4; ++w)
    for (int r = 0; r < 128; ++r)
      for (int c = 0; c < 8; ++c)
        out[(w * 128 + r) * 8 + c] = (int32_t)sg::cblock_lds_offset(w, r, c);
  return ok();
}

int gemm_lds_image_tile(int kind, const void* X, int64_t rows, int64_t row_bytes,
                        int64_t row0, int64_t byte0, void* out, void* stream) {
  const char* who = "gemm_lds_image_tile";
  if (kind < SG_IMG_HALF || kind > SG_IMG_CBLOCK)
    return fail(SG_ERR_DTYPE, "%s: unknown kind %d", who, kind);
  if (!X || !out) return fail(SG_ERR_NULL, "%s: X or out is NULL", who);
  if (!aligned16(X) || !aligned16(out) || row_bytes % 16)
    return fail(SG_ERR_ALIGN, "%s: X and out must be 16-byte aligned and row_bytes a "
                              "multiple of 16", who);
  if (rows <= 0 || row_bytes <= 0 || row0 < 0 || row0 >= rows || byte0 < 0 ||
      byte0 >= row_bytes || rows * row_bytes >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "%s: origin (%lld, %lld) outside the %lld x %lld operand", who,
                (long long)row0, (long long)byte0, (long long)rows, (long long)row_bytes);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const char* x = static_cast<const char*>(X);
  hipError_t e = hipSuccess;
  if (kind == SG_IMG_HALF || kind == SG_IMG_HALF_KEXACT) {
    if (byte0 % 128 || (kind == SG_IMG_HALF_KEXACT && row_bytes % 128))
      return fail(SG_ERR_SHAPE, "%s: byte0 %% 128 and (K-exact) row_bytes %% 128 must be 0",
                  who);
    const int64_t valid = rows - row0;
    e = sg::launch_lds_image_pp(kind, x + row0 * row_bytes, (uint32_t)(valid * row_bytes),
                                (uint32_t)row_bytes, (int)(valid < 256 ? valid : 256),
                                (uint32_t)byte0, (uint32_t)row_bytes, 32u, 0u, out, s);
  } else if (kind == SG_IMG_MN256) {
    if (row0 % 64 || byte0 % 256)
      return fail(SG_ERR_SHAPE, "%s: row0 %% 64 and byte0 %% 256 must be 0", who);
    const int64_t cols = (row_bytes - byte0) / 2;
    e = sg::launch_lds_image_pp(kind, x + byte0,
                                (uint32_t)((rows - 1) * row_bytes + (row_bytes - byte0)),
                                (uint32_t)row_bytes, (int)(cols < 256 ? cols : 256), 0u, 0u,
                                32u, (uint32_t)(row0 / 64), out, s);
  } else if (kind == SG_IMG_FP6) {
    if (row0 % 256 || byte0 % 96 || row_bytes % 96)
      return fail(SG_ERR_SHAPE, "%s: row0 %% 256, byte0 %% 96 and row_bytes %% 96 must be 0",
                  who);
    // As the MX kernel sets up a 256-row tile: below the operand's last tile
    // the descriptor covers the 8 bytes its shifted rows read past the tile;
    // in the last tile the rows at the last row's block position stay
    // unshifted.
    const int64_t left = rows - row0;
    const int m_valid = (int)(left < 256 ? left : 256);
    const uint32_t bytes = (uint32_t)(m_valid * row_bytes) + (left > 256 ? 8u : 0u);
    const uint32_t unshifted = left > 256 ? 32u : (uint32_t)((left - 1) & 31);
    e = sg::launch_lds_image_pp(kind, x + row0 * row_bytes, bytes, (uint32_t)row_bytes,
                                m_valid, 0u, 0u, unshifted, (uint32_t)(byte0 / 96), out, s);
  } else {
    if (row0 % 256 || byte0 % 512 || row_bytes / 2 > (int64_t{1} << 22))
      return fail(SG_ERR_SHAPE, "%s: row0 %% 256 and byte0 %% 512 must be 0 (and ldc <= "
                  "2^22)", who);
    const int64_t left = rows - row0, cols = (row_bytes - byte0) / 2;
    e = sg::launch_lds_image_cblock(X, row_bytes / 2, row0, byte0 / 2,
                                    (int)(left < 256 ? left : 256),
                                    (int)(cols < 256 ? cols : 256), out, s);
  }
  if (e != hipSuccess) return hip_fail(e, who);
  return ok();
}

int gemm_mfma_scale_probe(int fmt, const void* a, const void* b, const void* sa,
                          const void* sb, void* out, void* stream) {
  if (fmt != 0 && fmt != 2 && fmt != 3 && fmt != 4)
    return fail(SG_ERR_DTYPE, "gemm_mfma_scale_probe: fmt %d is not 0, 2, 3 or 4", fmt);
  if (!a || !b || !sa || !sb || !out)
    return fail(SG_ERR_NULL, "gemm_mfma_scale_probe: a NULL pointer");
  if (!aligned16(a) || !aligned16(b) || !aligned16(out))
    return fail(SG_ERR_ALIGN, "gemm_mfma_scale_probe: a, b and out must be 16-byte aligned");
  hipError_t e = sg::launch_mfma_scale_probe(fmt, a, b, sa, sb, out,
                                             static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "gemm_mfma_scale_probe launch");
  return ok();
}

int gemm_lds_image(const void* X, int64_t rows_total, int64_t K, int elem_bytes_,
                   int64_t row0, int64_t k0, int tile_rows, void* out, void* stream) {
  if (!X || !out) return fail(SG_ERR_NULL, "gemm_lds_image: X or out is NULL");
  if (elem_bytes_ != 1 && elem_bytes_ != 2)
    return fail(SG_ERR_DTYPE, "gemm_lds_image: elem_bytes must be 1 or 2");
  if (tile_rows != 128 && tile_rows != 256)
    return fail(SG_ERR_SHAPE, "gemm_lds_image: tile_rows must be 128 or 256");
  if (rows_total < 0 || K <= 0 || row0 < 0 || row0 >= rows_total || k0 < 0 || k0 >= K ||
      (k0 * elem_bytes_) % 128)
    return fail(SG_ERR_SHAPE, "gemm_lds_image: tile origin out of range or not on a "
                              "128-byte K boundary");
  if (!aligned16(X) || !aligned16(out) || (K * elem_bytes_) % 16)
    return fail(SG_ERR_ALIGN, "gemm_lds_image: 16-byte alignment required");
  if ((int64_t)tile_rows * K * elem_bytes_ >= kMaxExtent)
    return fail(SG_ERR_SHAPE, "gemm_lds_image: panel spans 2^31 bytes or more");
  hipError_t e = sg::launch_lds_image(X, rows_total, K, elem_bytes_, row0, k0, tile_rows,
                                      out, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "gemm_lds_image launch");
  return ok();
}

}  // extern "C"
