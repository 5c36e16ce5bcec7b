// efla_block_api.cu - the C ABI of the operators around the mixer (norm,
// short convolution, selective scan): validation, scratch sizing and kernel
// dispatch, as efla_api.cu has them for the mixer itself.
#include <cmath>

#include "efla_conv.cuh"
#include "efla_host.cuh"
#include "efla_norm.cuh"
#include "efla_scan_launch.cuh"

using namespace efla;
using namespace efla::host;
using scan::rows_in_vectors;

namespace {

constexpr int kMaxLength = 0x7fff0000;  // of a sequence: tiles past its end still count in 32 bits
constexpr long long kMaxBlocks = 0x7fff0000;  // of a grid: colsum_kernel's steps past the last of their rows still count in 32 bits

// One buffer of a call: where it is, how many bytes from its first to its last.
struct Buf {
    const void *p;
    size_t bytes;
};

// An output may not overlap an input or another output.
template <int NI, int NO> bool aliased(const Buf (&in)[NI], const Buf (&out)[NO]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return true;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
    }
    return false;
}

template <int N> bool all_aligned16(const void *const (&p)[N]) {
    for (const void *q : p)
        if (!aligned16(q)) return false;
    return true;
}

// Bytes that `rows` rows of `n` elements take, `ld` elements apart.
size_t extent(long long rows, long long ld, long long n, size_t e) {
    return rows > 0 ? ((size_t)(rows - 1) * ld + n) * e : 0;
}

size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

efla_status_t colsum(const float *part, int P, ColsumOut o, long long M, cudaStream_t st) {
    colsum_kernel<<<(unsigned)((M + 31) / 32), 1024, 0, st>>>(part, o, M, P);
    return launched();
}

// ---------------------------------------------------------------- norm

// Rows of up to 64 vectors share blocks of 256 threads; longer ones have a
// block of their own, of the whole warps that they need: with powers of two
// 16384 x 2048 in bf16 to 8 bits took 40.3 us (39.0 so), 21845 x 1536 46 (39),
// 6553 x 5120 75 (46).
template <typename T, typename R, int TPR, int IT, int RPI, bool ANY>
efla_status_t launch_norm_rows(const norm::FwdArgs &a, int nvec, cudaStream_t st) {
    const int threads = TPR > 0 ? norm::kThreadsOf<TPR> : (nvec + 32 * IT - 1) / (32 * IT) * 32;
    const long long rows = (long long)RPI * (TPR > 0 ? threads / TPR : 1);  // of a block
    // several rows in flight a thread once there are enough to fill the SMs
    if constexpr (RPI > 1)
        if (a.rows * threads < 512LL * num_sms() * rows) return launch_norm_rows<T, R, TPR, IT, 1, ANY>(a, nvec, st);
    norm::norm_fwd_kernel<T, R, TPR, IT, RPI, ANY><<<(unsigned)((a.rows + rows - 1) / rows), threads, 0, st>>>(a);
    return launched();
}

template <typename T, typename R, bool ANY> efla_status_t launch_norm_vectors(const norm::FwdArgs &a, int nvec, cudaStream_t st) {
    constexpr int R4 = ANY ? 1 : 4, R2 = ANY ? 1 : 2;
    if constexpr (!ANY) {
        if (nvec <= 16) return launch_norm_rows<T, R, 16, 1, R4, ANY>(a, nvec, st);
        if (nvec <= 32) return launch_norm_rows<T, R, 32, 1, R4, ANY>(a, nvec, st);
    }
    if (nvec <= 64) return launch_norm_rows<T, R, 32, 2, R2, ANY>(a, nvec, st);
    // two vectors a thread; four from 513 vectors on, for more blocks an SM (4096 x 8192, bf16 to bf16: 75 -> 72 us,
    // 6553 x 5120: 74 -> 66), but where the eight-bit output needs the registers (4096 x 8192: 54 -> 74)
    if (nvec <= (a.y8 ? 1024 : 512)) return launch_norm_rows<T, R, -512, 2, R2, ANY>(a, nvec, st);
    if (nvec <= 2048) return launch_norm_rows<T, R, -512, 4, 1, ANY>(a, nvec, st);
    if constexpr (sizeof(T) == 4) return launch_norm_rows<T, R, -512, 8, 1, ANY>(a, nvec, st);
    return EFLA_ERR_UNSUPPORTED;
}

template <typename T, typename R> efla_status_t launch_norm_fwd(const norm::FwdArgs &a, bool vec, cudaStream_t st) {
    constexpr int VEC = 16 / sizeof(T);
    if (vec) return launch_norm_vectors<T, R, false>(a, a.C / VEC, st);
    // vectors shifted to the row's alignment: up to VEC - 1 columns of the first and the last lie outside
    const int shifted = (a.C + 2 * (VEC - 1)) / VEC;
    if (a.C > 128 && shifted <= norm::kMaxC / VEC) return launch_norm_vectors<T, R, true>(a, shifted, st);
    if (a.C <= 128) norm::norm_fwd_any_kernel<T, R, 1, 1><<<(unsigned)((a.rows + 7) / 8), 256, 0, st>>>(a);
    else norm::norm_fwd_any_kernel<T, R, 16, 8><<<(unsigned)a.rows, 512, 0, st>>>(a);
    return launched();
}

// Blocks of the backward pass, each with a row of partial column sums: as
// many as are resident at once, fewer where there are fewer rows.
long long norm_bwd_blocks(long long rows) { return std::min<long long>(rows, 2LL * num_sms()); }

// Threads of a row and vectors of a thread for nvec vectors: two vectors a
// thread from 64 vectors on, so that the row's sums and root cost each
// element less, and up to 512 threads (with 1024 a thread has 64 registers
// and wide rows spill).  In fp32, rows of 513 to 1024 vectors have four a
// thread, and two blocks an SM (8192 x 4096: 95 -> 90 us); in bf16 that
// spills (4096 x 8192: 114 -> 177).
#define EFLA_NORM_VEC(LAUNCH, T, nvec)                                     \
    do {                                                                   \
        if ((nvec) <= 16) { LAUNCH(16, 1); }                               \
        else if ((nvec) <= 32) { LAUNCH(32, 1); }                          \
        else if ((nvec) <= 64) { LAUNCH(32, 2); }                          \
        else if ((nvec) <= 128) { LAUNCH(64, 2); }                         \
        else if ((nvec) <= 256) { LAUNCH(128, 2); }                        \
        else if ((nvec) <= 512) { LAUNCH(256, 2); }                        \
        else if ((nvec) <= 1024) { LAUNCH((sizeof(T) == 4 ? 256 : 512), (sizeof(T) == 4 ? 4 : 2)); } \
        else if ((nvec) <= 2048) { LAUNCH(512, 4); }                       \
        else if constexpr (sizeof(T) == 4) { LAUNCH(512, 8); }             \
    } while (0)

// Warps of a row and groups of 128 columns of a warp, for any width.
#define EFLA_NORM_ANY(LAUNCH, C)                         \
    do {                                                 \
        if ((C) <= 128) { LAUNCH(1, 1); }                \
        else if ((C) <= 512) { LAUNCH(1, 4); }           \
        else if ((C) <= 2048) { LAUNCH(4, 4); }          \
        else if ((C) <= 8192) { LAUNCH(16, 4); }         \
        else { LAUNCH(16, 8); }                          \
    } while (0)

template <typename T, typename R> efla_status_t launch_norm_bwd(const norm::BwdArgs &a, bool vec, int blocks, cudaStream_t st) {
    constexpr int VEC = 16 / sizeof(T);
    if (!vec) {
#define EFLA_L(WPR, IT) norm::norm_bwd_any_kernel<T, R, WPR, IT><<<blocks, norm::kThreadsOf<WPR * 32>, 0, st>>>(a)
        EFLA_NORM_ANY(EFLA_L, a.C);
#undef EFLA_L
        return launched();
    }
    const int nvec = a.C / VEC;
#define EFLA_L(TPR, IT) \
    norm::norm_bwd_kernel<T, R, TPR, IT, (IT == 1 || (IT == 2 && sizeof(T) == 4) ? 2 : 1)><<<blocks, norm::kThreadsOf<TPR>, 0, st>>>(a)
    EFLA_NORM_VEC(EFLA_L, T, nvec);
#undef EFLA_L
    return launched();
}

// ---------------------------------------------------------------- conv

#define EFLA_CONV_K(KERNEL, T, VEC, K, GRID, BLOCK, ...)                                            \
    do {                                                                                            \
        if ((K) == 2) KERNEL<T, 2, VEC><<<GRID, BLOCK, 0, st>>>(__VA_ARGS__);                       \
        else if ((K) == 3) KERNEL<T, 3, VEC><<<GRID, BLOCK, 0, st>>>(__VA_ARGS__);                  \
        else KERNEL<T, 4, VEC><<<GRID, BLOCK, 0, st>>>(__VA_ARGS__);                                \
    } while (0)

int conv_tiles(int L, int run) {
    const int n = run * conv::kWarps;
    return L > 0 ? (L + n - 1) / n : 1;
}

// Channels of a thread in the backward pass: pairs, where every row of x and
// of y (whose rows are a head's where there are heads) begins on one.
int conv_bwd_channels(const void *x, long long ldx, int C, int heads, size_t e) {
    return (heads ? C / heads : C) % 2 == 0 && rows_in_vectors(x, ldx, 2, e) ? 2 : 1;
}

// Tokens of a thread's run in the backward pass, a power of two: long runs
// recompute and add up less, short ones give a short or narrow input enough
// threads.  The cost of a choice is counted in the waves of its blocks, four an
// SM of pairs and five of single channels, as their registers allow; a wave
// takes its runs' tokens and a start of 24 more, and a part of a wave, bound by
// latency, no less than 0.7 of one.  Where there are lengths, which the host does
// not see, blocks past a sequence's end do nothing and long ones are half idle:
// four fifths of the blocks are counted and runs end at 128.  Over 230 sizes of 1
// to 32 sequences, the run so taken is 0.7% slower than the fastest in the mean
// (17% at most), with random lengths 5% (30%), with lengths all whole 4% (27%).
// Runs of 8, 16, 32, 64, 128 and 256, in us:
//   pairs    4 x 4096 x 2048, bf16    -   -  86  72  65  61     32 x 100 x 2048, bf16  52  38  28  31  39  39
//            1 x 16384 x 1024, fp32   -   -  50  45  41  49     18 x 22 x 3584, bf16   19  19  23  23  23  23
//   singles  8 x 2047 x 1001, fp32    -   -  59  54  57  53     8 x 4096 x 1001, fp32   -   - 110 101  96 105
//            16 x 1000 x 2050 of odd heads, fp32  -  -  108  98  91  99
int conv_run(int B, int L, int C, int channels, bool lengths) {
    const int cols = (C + 32 * channels - 1) / (32 * channels);
    const double wave = (channels == 2 ? 4.0 : 5.0) * num_sms(), share = lengths ? 0.8 : 1.0;
    int best = conv::kShortRun;
    double least = 1e300;
    for (int r = lengths ? conv::kLongRun / 2 : conv::kLongRun; r >= conv::kShortRun; r /= 2) {
        const double waves = share * B * conv_tiles(L, r) * cols / wave, part = waves - std::floor(waves);
        const double cost = (r + 24) * (std::floor(waves) + (part > 0 ? std::max(part, 0.7) : 0.0));
        if (cost < least) least = cost, best = r;
    }
    return best;
}

// The forward pass stands on the SMs in waves of four blocks each (eight of
// single channels), so of the runs the one whose waves are shortest, each with
// its start counted as eight tokens: 4 x 4096 x 2048, bf16, 576 blocks with runs
// of 120 29.5 us, 512 with 128 30.1, two waves with 112 35.7 and with 64 32.5.
int conv_fwd_run(int B, int L, int cols, bool vec) {
    const double wave = (vec ? 4.0 : 8.0) * num_sms();
    int best = conv::kLongFwdRun;
    double least = 1e300;
    for (int r = conv::kLongFwdRun; r >= conv::kShortRun; r -= conv::kAhead) {
        const double cost = std::ceil((double)B * conv_tiles(L, r) * cols / wave) * (r + conv::kAhead);
        if (cost < least) least = cost, best = r;
    }
    return best;
}

efla_status_t check_conv(efla_dtype_t dtype, long long ldx, int B, int L, int C, int K, int heads) {
    if (!known_dtype(dtype)) return EFLA_ERR_DTYPE;
    if (B < 0 || L < 0 || L > kMaxLength || C < 0 || heads < 0 || K <= 0) return EFLA_ERR_SHAPE;
    if (K < 2 || K > 4) return EFLA_ERR_UNSUPPORTED;
    if (heads && C % heads) return EFLA_ERR_SHAPE;
    if (ldx < C || ldx > kMaxElems) return EFLA_ERR_SHAPE;
    if ((double)B * (L + 4.0) * (double)ldx > (double)kMaxElems) return EFLA_ERR_SHAPE;
    if ((long long)B * conv_tiles(L, conv::kShortRun) > kMaxBlocks || C > 65535 * 32) return EFLA_ERR_SHAPE;
    return EFLA_OK;
}

// ---------------------------------------------------------------- scan

// How the work is cut.  A block's recurrence is four warps, one a scheduler,
// which alone leaves most of its latencies open, so few blocks want short work
// a token (two state values a lane) and many want little shared memory traffic
// a value (two channels a lane).  us in the order of the kinds below:
//   forward  1 x 4096 x 2048 x 16   91  157  278   segments 109 to 118
//            2 x 4096 x 2048 x 16  165  173  337
//            8 x 2048 x 1024 x 16  164  137  173
//           16 x 1024 x 4096 x 16  564  457  444
//            2 x 2048 x 1024 x 64  138  138  119
//   backward 2 x 4096 x 2048 x 16  707  842
//            8 x 2048 x 1024 x 16  676  550
// Segments pay for a second pass over the exponentials, so they stand where
// that fills idle SMs: 1 x 16384 x 512 x 16 396 -> 107 us, backward 2079 -> 344;
// 1 x 4096 x 2048 x 16 backward 589 -> 380, where forward is better off whole.
scan::Plan scan_plan(int B, int L, int C, int G, int N, bool bwd) {
    scan::Plan p;
    const int sms = num_sms(), cg = C / G;
    // 0: one channel and two state values a lane (four of 64); 1: four; 2: two channels, four values each (two of 8)
    const auto shape = [&](int kind) {
        p.ns = N == 64 || (kind > 0 && !(N == 8 && kind == 2)) ? 4 : 2;
        p.cp = kind == 2 ? 2 : 1;
        const int ct = scan::tile_channels(N, p.ns, p.cp);
        p.tpg = (cg + ct - 1) / ct;
        return p.blocks = (long long)B * G * p.tpg;
    };
    p.nseg = 1;
    const long long two = shape(2), one = shape(1), zero = shape(0);
    if (N == 64 ? two * 2 >= sms : two >= 3 * sms && !(bwd && N < 32)) {
        shape(2);
    } else if (one >= sms) {
        shape(1);
    } else if (zero * 3 < sms * (bwd ? 4LL : 2LL) && L >= 3 * 128) {
        shape(1);
        p.nseg = (int)std::max<long long>(1, std::min<long long>(4LL * sms / one, L / 128));
    }
    const int seg = (L + p.nseg - 1) / p.nseg;
    p.seg = (seg + 31) / 32 * 32;  // 32: a multiple of every tile
    p.nseg = L > 0 ? (L + p.seg - 1) / p.seg : 1;
    return p;
}

size_t seg_floats(const scan::Plan &p, int B, int C, int N, bool bwd) {
    if (p.nseg == 1) return 0;
    const size_t bc = (size_t)B * C;
    return bc * N * (p.nseg * (bwd ? 2 : 1) + 1) + round16(bc * p.nseg * 4) / 4;
}

void carve_segments(scan::Args &a, float *&ws, bool bwd) {
    if (a.nseg == 1) return;
    const size_t bc = (size_t)a.B * a.C;
    a.seg_h = ws;
    ws += bc * a.N * a.nseg;
    a.seg_0 = ws;
    ws += bc * a.N;
    if (bwd) {
        a.seg_p = ws;
        ws += bc * a.N * a.nseg;
    }
    a.seg_d = ws;
    ws += round16(bc * a.nseg * 4) / 4;
}

struct BwdSizes {
    size_t seg, ckpt, bc, part;
    size_t bytes() const { return (seg + ckpt + bc + part) * sizeof(float); }
};
BwdSizes bwd_sizes(const scan::Plan &p, int B, int L, int C, int G, int N) {
    BwdSizes s;
    s.seg = seg_floats(p, B, C, N, true);
    s.ckpt = (size_t)p.blocks * p.nseg * (p.seg / p.sub()) * scan::kThreads * p.ns * p.cp;
    s.bc = (size_t)p.tpg * B * L * G * 2 * N;
    s.part = (size_t)p.nseg * B * C * (N + 2);
    return s;
}

efla_status_t check_scan(efla_dtype_t dtype, int B, int L, int C, int G, int N) {
    if (!known_dtype(dtype)) return EFLA_ERR_DTYPE;
    if (B < 0 || L < 0 || L > kMaxLength || C < 0 || G <= 0 || N <= 0) return EFLA_ERR_SHAPE;
    if (N != 8 && N != 16 && N != 32 && N != 64) return EFLA_ERR_UNSUPPORTED;
    if (C % G) return EFLA_ERR_SHAPE;
    if ((double)B * (L + 1.0) * C > (double)kMaxElems || (double)B * (L + 1.0) * G * N > (double)kMaxElems ||
        (double)B * C * N > (double)kMaxElems / 64)
        return EFLA_ERR_SHAPE;
    if ((double)C * N > 2147483647.0) return EFLA_ERR_SHAPE;  // a sequence's state values are counted in 32 bits
    return EFLA_OK;
}

// Whether a grid holds a pass's blocks.
bool scan_fits(const scan::Plan &p) { return p.blocks * p.nseg <= kMaxBlocks; }

template <typename T> efla_status_t run_scan_fwd(const scan::Args &a, const scan::Plan &p, cudaStream_t st) {
    if (p.nseg > 1) {
        const efla_status_t s = scan::launch_forward<T>(scan::STATE, a, p, st);
        if (s != EFLA_OK) return s;
    }
    return scan::launch_forward<T>(scan::FULL, a, p, st);
}

template <typename T>
efla_status_t run_scan_bwd(const scan::Args &a, const scan::Plan &p, void *dB, void *dC, float *dA, float *dD,
                           float *db, cudaStream_t st) {
    efla_status_t s = EFLA_OK;
    if (p.nseg > 1) {
        s = scan::launch_forward<T>(scan::STATE, a, p, st);
        if (s == EFLA_OK) s = scan::launch_forward<T>(scan::BACK, a, p, st);
    }
    if (s == EFLA_OK) s = scan::launch_backward<T>(a, p, st);
    if (s != EFLA_OK) return s;
    const long long rows = (long long)a.B * a.L * a.G, quads = rows * 2 * a.N / 4;
    scan::scan_bc_kernel<T><<<(unsigned)((quads + 255) / 256), 256, 0, st>>>(a.part_bc, static_cast<T *>(dB),
                                                                          static_cast<T *>(dC), rows, a.N, a.tpg);
    if (launched() != EFLA_OK) return EFLA_ERR_CUDA;
    const long long cn = (long long)a.C * a.N;
    return colsum(a.part, a.nseg * a.B, ColsumOut{{dA, dD, db}, {cn, cn + a.C, cn + 2 * a.C}}, cn + 2 * a.C, st);
}

template <typename T, int N> efla_status_t launch_scan_step(scan::Args a, cudaStream_t st) {
    a.vec = rows_in_vectors(a.Bm, a.ldb, 8, sizeof(T)) && rows_in_vectors(a.Cm, a.ldc, 8, sizeof(T));
    const long long gx = ((long long)a.C * (N / 8) + 127) / 128;
    scan::scan_step_kernel<T, N><<<dim3((unsigned)gx, a.B), 128, 0, st>>>(a);
    return launched();
}

}  // namespace

extern "C" {

efla_status_t efla_norm_fwd(const void *x, efla_dtype_t dtype, const void *res, efla_dtype_t res_dtype,
                            const float *weight, float eps, void *y, void *y8, float *scale, int group, void *res_out,
                            long long rows, int C, efla_stream_t stream) {
    NvtxRange nvtx_("efla_norm_fwd");
    if (!known_dtype(dtype) || !known_dtype(res_dtype)) return EFLA_ERR_DTYPE;
    if (rows < 0 || C < 0) return EFLA_ERR_SHAPE;
    if (res && res_dtype == EFLA_BF16 && dtype == EFLA_F32) return EFLA_ERR_UNSUPPORTED;
    if (C > norm::kMaxC || (group != 0 && group != norm::kGroup)) return EFLA_ERR_UNSUPPORTED;
    if ((double)rows * C > (double)kMaxElems || rows > 0x7fffffffLL) return EFLA_ERR_SHAPE;
    if (rows == 0 || C == 0) return EFLA_OK;
    if (!x || !weight || (!y && !y8) || (y8 && !scale) || (res_out && !res)) return EFLA_ERR_NULL;
    if (!all_aligned16({x, res, weight, y, y8, scale, res_out})) return EFLA_ERR_ALIGN;
    const size_t n = (size_t)rows * C, xb = n * esize(dtype), rb = n * esize(res_dtype);
    const size_t sb = (size_t)rows * (group ? (C + group - 1) / group : 1) * sizeof(float);
    // in place: res_out on res, and y or res_out on x where the types agree
    const bool same = dtype == res_dtype;
    const Buf in[] = {{x, xb}, {res, rb}, {weight, (size_t)C * 4}};
    const Buf out[] = {{y == x ? nullptr : y, xb}, {y8, n}, {scale, sb}, {res_out == res || (res_out == x && same) ? nullptr : res_out, rb}};
    if (aliased(in, out)) return EFLA_ERR_ALIAS;
    if (y == x && (overlaps(y, xb, res, rb) || overlaps(y, xb, y8, n) || overlaps(y, xb, scale, sb))) return EFLA_ERR_ALIAS;
    if (res_out && (res_out == res || res_out == x) &&
        (overlaps(res_out, rb, y, xb) || overlaps(res_out, rb, y8, n) || overlaps(res_out, rb, scale, sb) ||
         (res_out == res ? overlaps(res, rb, x, xb) : overlaps(x, xb, res, rb))))
        return EFLA_ERR_ALIAS;
    const norm::FwdArgs a{x, res, weight, y, res_out, static_cast<unsigned char *>(y8), scale, eps, 1.f / C, group, C, rows};
    const bool vec = C % (16 / (int)esize(dtype)) == 0;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == EFLA_F32) return launch_norm_fwd<float, float>(a, vec, st);
    if (res && res_dtype == EFLA_F32) return launch_norm_fwd<__nv_bfloat16, float>(a, vec, st);
    return launch_norm_fwd<__nv_bfloat16, __nv_bfloat16>(a, vec, st);
}

size_t efla_norm_bwd_workspace_size(long long rows, int C) {
    if (rows <= 0 || C <= 0 || C > norm::kMaxC) return 0;
    return round16((size_t)norm_bwd_blocks(rows) * C * sizeof(float));
}

efla_status_t efla_norm_bwd(const void *dy, efla_dtype_t dtype, const void *h, efla_dtype_t h_dtype,
                            const float *weight, float eps, const void *dres_out, void *dx, void *dres, float *dweight,
                            long long rows, int C, void *workspace, size_t workspace_bytes, efla_stream_t stream) {
    NvtxRange nvtx_("efla_norm_bwd");
    if (!known_dtype(dtype) || !known_dtype(h_dtype)) return EFLA_ERR_DTYPE;
    if (rows < 0 || C < 0) return EFLA_ERR_SHAPE;
    if ((h_dtype == EFLA_BF16 && dtype == EFLA_F32) || C > norm::kMaxC) return EFLA_ERR_UNSUPPORTED;
    if ((double)rows * C > (double)kMaxElems || rows > 0x7fffffffLL) return EFLA_ERR_SHAPE;
    if (C == 0) return EFLA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!dweight) return EFLA_ERR_NULL;
    if (!aligned16(dweight)) return EFLA_ERR_ALIGN;
    if (rows == 0)  // no rows: their sum is zero
        return cudaMemsetAsync(dweight, 0, C * sizeof(float), st) == cudaSuccess ? EFLA_OK : EFLA_ERR_CUDA;
    if (!dy || !h || !weight || (!dx && !dres)) return EFLA_ERR_NULL;
    if (!all_aligned16({dy, h, weight, dres_out, dx, dres, workspace})) return EFLA_ERR_ALIGN;
    const size_t n = (size_t)rows * C, need = efla_norm_bwd_workspace_size(rows, C);
    if (!workspace || workspace_bytes < need) return EFLA_ERR_WORKSPACE;
    const Buf in[] = {{dy, n * esize(dtype)}, {h, n * esize(h_dtype)}, {weight, (size_t)C * 4}, {dres_out, n * esize(h_dtype)}};
    const Buf out[] = {{dx, n * esize(dtype)}, {dres, n * esize(h_dtype)}, {dweight, (size_t)C * 4}, {workspace, need}};
    if (aliased(in, out)) return EFLA_ERR_ALIAS;
    float *part = static_cast<float *>(workspace);
    const norm::BwdArgs a{dy, h, dres_out, weight, dx, dres, part, eps, 1.f / C, C, rows};
    const int blocks = (int)norm_bwd_blocks(rows);
    const bool vec = C % (16 / (int)esize(dtype)) == 0;
    efla_status_t s;
    if (dtype == EFLA_F32) s = launch_norm_bwd<float, float>(a, vec, blocks, st);
    else if (h_dtype == EFLA_F32) s = launch_norm_bwd<__nv_bfloat16, float>(a, vec, blocks, st);
    else s = launch_norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, vec, blocks, st);
    if (s != EFLA_OK) return s;
    return colsum(part, blocks, ColsumOut{{dweight, nullptr, nullptr}, {C, C, C}}, C, st);
}

efla_status_t efla_conv_fwd(const void *x, long long ldx, efla_dtype_t dtype, const float *weight, const float *bias,
                            const void *state, const int *lengths, int silu, void *y, int heads, void *state_out,
                            int B, int L, int C, int K, efla_stream_t stream) {
    NvtxRange nvtx_("efla_conv_fwd");
    efla_status_t s = check_conv(dtype, ldx, B, L, C, K, heads);
    if (s != EFLA_OK) return s;
    if (B == 0 || C == 0 || (L == 0 && !state_out)) return EFLA_OK;
    const size_t e = esize(dtype);
    if ((L > 0 && (!x || !y)) || !weight) return EFLA_ERR_NULL;
    if (!aligned_to(x, e) || !aligned_to(lengths, 4) || !all_aligned16({weight, bias, state, y, state_out}))
        return EFLA_ERR_ALIGN;
    const size_t yb = (size_t)B * L * C * e, sb = (size_t)B * (K - 1) * C * e;
    const size_t xb = extent((long long)B * L, ldx, C, e);
    const Buf in[] = {{x, xb}, {weight, (size_t)C * K * 4}, {bias, (size_t)C * 4}, {lengths, (size_t)B * 4},
                      {state == state_out ? nullptr : state, sb}};
    const Buf out[] = {{y, yb}, {state_out, sb}};
    if (aliased(in, out) || overlaps(y, yb, state, sb)) return EFLA_ERR_ALIAS;
    conv::Args a{};
    a.x = x; a.ldx = ldx; a.w = weight; a.bias = bias; a.state = state; a.lengths = lengths; a.silu = silu;
    a.head = heads ? C / heads : 0;
    const int row = heads ? C / heads : C, VEC = 4;
    const bool vec = row % VEC == 0 && rows_in_vectors(x, ldx, VEC, e);
    const int cols = (C + 32 * (vec ? VEC : 1) - 1) / (32 * (vec ? VEC : 1));
    a.B = B; a.L = L; a.C = C; a.run = conv_fwd_run(B, L, cols, vec); a.tiles = conv_tiles(L, a.run);
    a.y = y; a.state_out = state_out;
    const dim3 grid((unsigned)(B * a.tiles), (unsigned)cols);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == EFLA_F32) {
        if (vec) EFLA_CONV_K(conv::conv_fwd_kernel, float, 4, K, grid, 32 * conv::kWarps, a);
        else EFLA_CONV_K(conv::conv_fwd_kernel, float, 1, K, grid, 32 * conv::kWarps, a);
    } else {
        if (vec) EFLA_CONV_K(conv::conv_fwd_kernel, __nv_bfloat16, 4, K, grid, 32 * conv::kWarps, a);
        else EFLA_CONV_K(conv::conv_fwd_kernel, __nv_bfloat16, 1, K, grid, 32 * conv::kWarps, a);
    }
    return launched();
}

size_t efla_conv_bwd_workspace_size(int B, int L, int C, int K) {
    if (B <= 0 || L < 0 || L > kMaxLength || C <= 0 || K < 2 || K > 4) return 0;
    int tiles = 0;  // whichever way the rows turn out to be read, with lengths or without
    for (int channels = C % 2 ? 1 : 2; channels > 0; --channels)
        for (bool lengths : {false, true}) tiles = std::max(tiles, conv_tiles(L, conv_run(B, L, C, channels, lengths)));
    return round16((size_t)B * tiles * C * (K + 1) * sizeof(float));
}

efla_status_t efla_conv_bwd(const void *dy, const void *x, long long ldx, efla_dtype_t dtype, const float *weight,
                            const float *bias, const void *state, const int *lengths, int silu, int heads,
                            const void *dstate_out, void *dx, float *dweight, float *dbias, void *dstate, int B, int L,
                            int C, int K, void *workspace, size_t workspace_bytes, efla_stream_t stream) {
    NvtxRange nvtx_("efla_conv_bwd");
    efla_status_t s = check_conv(dtype, ldx, B, L, C, K, heads);
    if (s != EFLA_OK) return s;
    if (C == 0) return EFLA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t e = esize(dtype);
    if (!dweight) return EFLA_ERR_NULL;
    if (!aligned16(dweight) || !aligned16(dbias)) return EFLA_ERR_ALIGN;
    if (B == 0) {  // no sequences: the sums are zero
        if (cudaMemsetAsync(dweight, 0, (size_t)C * K * 4, st) != cudaSuccess) return EFLA_ERR_CUDA;
        return !dbias || cudaMemsetAsync(dbias, 0, (size_t)C * 4, st) == cudaSuccess ? EFLA_OK : EFLA_ERR_CUDA;
    }
    if ((L > 0 && (!dy || !x || !dx)) || !weight) return EFLA_ERR_NULL;
    if (!aligned_to(x, e) || !aligned_to(lengths, 4) ||
        !all_aligned16({dy, weight, bias, state, dstate_out, dx, dstate, workspace}))
        return EFLA_ERR_ALIGN;
    const size_t need = efla_conv_bwd_workspace_size(B, L, C, K);
    if (!workspace || workspace_bytes < need) return EFLA_ERR_WORKSPACE;
    const size_t yb = (size_t)B * L * C * e, sb = (size_t)B * (K - 1) * C * e;
    const Buf in[] = {{dy, yb}, {x, extent((long long)B * L, ldx, C, e)}, {weight, (size_t)C * K * 4},
                      {bias, (size_t)C * 4}, {lengths, (size_t)B * 4}, {state, sb}, {dstate_out, sb}};
    const Buf out[] = {{dx, yb}, {dweight, (size_t)C * K * 4}, {dbias, (size_t)C * 4}, {dstate, sb}, {workspace, need}};
    if (aliased(in, out)) return EFLA_ERR_ALIAS;
    conv::Args a{};
    a.x = x; a.ldx = ldx; a.w = weight; a.bias = bias; a.state = state; a.lengths = lengths; a.silu = silu;
    a.head = heads ? C / heads : 0;
    const int channels = conv_bwd_channels(x, ldx, C, heads, e);
    a.B = B; a.L = L; a.C = C; a.run = conv_run(B, L, C, channels, lengths != nullptr); a.tiles = conv_tiles(L, a.run);
    a.dy = dy; a.dstate_out = dstate_out; a.dx = dx; a.dstate = dstate;
    const long long P = (long long)B * a.tiles;
    a.part = static_cast<float *>(workspace);
    const bool vec = channels == 2;
    const dim3 grid((unsigned)P, (unsigned)((C + 32 * channels - 1) / (32 * channels)));
    if (dtype == EFLA_F32) {
        if (vec) EFLA_CONV_K(conv::conv_bwd_kernel, float, 2, K, grid, 32 * conv::kWarps, a);
        else EFLA_CONV_K(conv::conv_bwd_kernel, float, 1, K, grid, 32 * conv::kWarps, a);
    } else {
        if (vec) EFLA_CONV_K(conv::conv_bwd_kernel, __nv_bfloat16, 2, K, grid, 32 * conv::kWarps, a);
        else EFLA_CONV_K(conv::conv_bwd_kernel, __nv_bfloat16, 1, K, grid, 32 * conv::kWarps, a);
    }
    if (launched() != EFLA_OK) return EFLA_ERR_CUDA;
    const long long M = (long long)C * K;
    return colsum(a.part, (int)P, ColsumOut{{dweight, dbias, nullptr}, {M, M + C, M + C}}, M + C, st);
}

efla_status_t efla_conv_step(const void *x, long long ldx, efla_dtype_t dtype, void *state, const float *weight,
                             const float *bias, int silu, void *y, int B, int C, int K, efla_stream_t stream) {
    NvtxRange nvtx_("efla_conv_step");
    efla_status_t s = check_conv(dtype, ldx, B, 1, C, K, 0);
    if (s != EFLA_OK) return s;
    if (B == 0 || C == 0) return EFLA_OK;
    if (!x || !state || !weight || !y) return EFLA_ERR_NULL;
    const size_t e = esize(dtype);
    if (!aligned_to(x, e) || !all_aligned16({state, weight, bias, y})) return EFLA_ERR_ALIGN;
    const Buf in[] = {{x, extent(B, ldx, C, e)}, {weight, (size_t)C * K * 4}, {bias, (size_t)C * 4}};
    const Buf out[] = {{state, (size_t)B * (K - 1) * C * e}, {y, (size_t)B * C * e}};
    if (aliased(in, out)) return EFLA_ERR_ALIAS;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // two channels a thread: at decode batches the launch is latency, so threads are spread over the SMs
    const bool vec = C % 2 == 0 && rows_in_vectors(x, ldx, 2, e);
    const dim3 grid((unsigned)B, (unsigned)((C + 128 * (vec ? 2 : 1) - 1) / (128 * (vec ? 2 : 1))));
    if (dtype == EFLA_F32) {
        const float *xp = static_cast<const float *>(x);
        float *sp = static_cast<float *>(state), *yp = static_cast<float *>(y);
        if (vec) EFLA_CONV_K(conv::conv_step_kernel, float, 2, K, grid, 128, xp, ldx, sp, weight, bias, yp, silu, C);
        else EFLA_CONV_K(conv::conv_step_kernel, float, 1, K, grid, 128, xp, ldx, sp, weight, bias, yp, silu, C);
    } else {
        const __nv_bfloat16 *xp = static_cast<const __nv_bfloat16 *>(x);
        __nv_bfloat16 *sp = static_cast<__nv_bfloat16 *>(state), *yp = static_cast<__nv_bfloat16 *>(y);
        if (vec) EFLA_CONV_K(conv::conv_step_kernel, __nv_bfloat16, 2, K, grid, 128, xp, ldx, sp, weight, bias, yp, silu, C);
        else EFLA_CONV_K(conv::conv_step_kernel, __nv_bfloat16, 1, K, grid, 128, xp, ldx, sp, weight, bias, yp, silu, C);
    }
    return launched();
}

int efla_diag_conv_run(int B, int L, int C, int channels, int backward, int lengths) {
    if (B <= 0 || L <= 0 || L > kMaxLength || C <= 0 || (channels != 1 && channels != (backward ? 2 : 4))) return 0;
    return backward ? conv_run(B, L, C, channels, lengths != 0) : conv_fwd_run(B, L, (C + 32 * channels - 1) / (32 * channels), channels > 1);
}

size_t efla_scan_fwd_workspace_size(int B, int L, int C, int G, int N) {
    if (B <= 0 || L <= 0 || C <= 0 || check_scan(EFLA_F32, B, L, C, G, N) != EFLA_OK) return 0;
    const scan::Plan p = scan_plan(B, L, C, G, N, false);
    return scan_fits(p) ? seg_floats(p, B, C, N, false) * sizeof(float) : 0;
}

efla_status_t efla_diag_scan_plan(int B, int L, int C, int G, int N, int backward, int plan[5]) {
    const efla_status_t s = check_scan(EFLA_F32, B, L, C, G, N);
    if (s != EFLA_OK) return s;
    if (!plan) return EFLA_ERR_NULL;
    if (B == 0 || L == 0 || C == 0) return EFLA_ERR_SHAPE;
    const scan::Plan p = scan_plan(B, L, C, G, N, backward != 0);
    if (!scan_fits(p)) return EFLA_ERR_SHAPE;
    plan[0] = p.ns; plan[1] = p.cp; plan[2] = p.nseg; plan[3] = p.seg; plan[4] = p.tpg;
    return EFLA_OK;
}

efla_status_t efla_scan_fwd(const void *x, long long ldx, const void *dt, long long lddt, const float *A,
                            const void *Bm, long long ldb, const void *Cm, long long ldc, const float *D, const void *z,
                            long long ldz, const float *dt_bias, const float *h0, const int *lengths,
                            efla_dtype_t dtype, int softplus, void *y, float *h_L, int B, int L, int C, int G, int N,
                            void *workspace, size_t workspace_bytes, efla_stream_t stream) {
    NvtxRange nvtx_("efla_scan_fwd");
    efla_status_t s = check_scan(dtype, B, L, C, G, N);
    if (s != EFLA_OK) return s;
    if (B == 0 || C == 0) return EFLA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t e = esize(dtype), hb = (size_t)B * C * N * sizeof(float);
    if (L == 0) {  // empty sequence: the state passes through unchanged
        if (!h_L || h_L == h0) return EFLA_OK;
        if (!aligned16(h_L) || !aligned16(h0)) return EFLA_ERR_ALIGN;
        if (overlaps(h_L, hb, h0, hb)) return EFLA_ERR_ALIAS;
        const cudaError_t r = h0 ? cudaMemcpyAsync(h_L, h0, hb, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(h_L, 0, hb, st);
        return r == cudaSuccess ? EFLA_OK : EFLA_ERR_CUDA;
    }
    if (ldx < C || lddt < C || (z && ldz < C) || ldb < (long long)G * N || ldc < (long long)G * N) return EFLA_ERR_SHAPE;
    if ((double)B * L * std::max({ldx, lddt, z ? ldz : 0, ldb, ldc}) > (double)kMaxElems) return EFLA_ERR_SHAPE;
    const scan::Plan p = scan_plan(B, L, C, G, N, false);
    if (!scan_fits(p)) return EFLA_ERR_SHAPE;
    if (!x || !dt || !A || !Bm || !Cm || !y) return EFLA_ERR_NULL;
    if (!aligned_to(x, e) || !aligned_to(dt, e) || !aligned_to(Bm, e) || !aligned_to(Cm, e) || !aligned_to(z, e) ||
        !aligned_to(lengths, 4) || !all_aligned16({A, D, dt_bias, h0, y, h_L, workspace}))
        return EFLA_ERR_ALIGN;
    const size_t need = seg_floats(p, B, C, N, false) * sizeof(float);
    if (need && (!workspace || workspace_bytes < need)) return EFLA_ERR_WORKSPACE;
    const long long rows = (long long)B * L;
    const Buf in[] = {{x, extent(rows, ldx, C, e)}, {dt, extent(rows, lddt, C, e)}, {z, extent(rows, ldz, C, e)},
                      {Bm, extent(rows, ldb, (long long)G * N, e)}, {Cm, extent(rows, ldc, (long long)G * N, e)},
                      {A, (size_t)C * N * 4}, {D, (size_t)C * 4}, {dt_bias, (size_t)C * 4}, {lengths, (size_t)B * 4},
                      {h0 == h_L ? nullptr : h0, hb}};
    const Buf out[] = {{y, (size_t)rows * C * e}, {h_L, hb}, {need ? workspace : nullptr, need}};
    if (aliased(in, out) || overlaps(y, (size_t)rows * C * e, h0, hb) || overlaps(workspace, need, h0, hb)) return EFLA_ERR_ALIAS;
    scan::Args a{};
    a.x = x; a.dt = dt; a.z = z; a.Bm = Bm; a.Cm = Cm;
    a.ldx = ldx; a.lddt = lddt; a.ldz = ldz; a.ldb = ldb; a.ldc = ldc;
    a.A = A; a.D = D; a.dt_bias = dt_bias; a.h0 = h0; a.lengths = lengths; a.y = y; a.h_L = h_L; a.softplus = softplus;
    a.B = B; a.L = L; a.C = C; a.G = G; a.N = N; a.tpg = p.tpg; a.nseg = p.nseg; a.seg = p.seg;
    float *ws = static_cast<float *>(workspace);
    carve_segments(a, ws, false);
    return dtype == EFLA_F32 ? run_scan_fwd<float>(a, p, st) : run_scan_fwd<__nv_bfloat16>(a, p, st);
}

size_t efla_scan_bwd_workspace_size(int B, int L, int C, int G, int N) {
    if (B <= 0 || L <= 0 || C <= 0 || check_scan(EFLA_F32, B, L, C, G, N) != EFLA_OK) return 0;
    const scan::Plan p = scan_plan(B, L, C, G, N, true);
    return scan_fits(p) ? bwd_sizes(p, B, L, C, G, N).bytes() : 0;
}

efla_status_t efla_scan_bwd(const void *dy, const void *x, long long ldx, const void *dt, long long lddt,
                            const float *A, const void *Bm, long long ldb, const void *Cm, long long ldc,
                            const float *D, const void *z, long long ldz, const float *dt_bias, const float *h0,
                            const int *lengths, const float *dh_L, efla_dtype_t dtype, int softplus, void *dx,
                            void *ddt, float *dA, void *dB, void *dC, float *dD, void *dz, float *ddt_bias, float *dh0,
                            int B, int L, int C, int G, int N, void *workspace, size_t workspace_bytes,
                            efla_stream_t stream) {
    NvtxRange nvtx_("efla_scan_bwd");
    efla_status_t s = check_scan(dtype, B, L, C, G, N);
    if (s != EFLA_OK) return s;
    if (C == 0) return EFLA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t e = esize(dtype), hb = (size_t)B * C * N * sizeof(float), pb = (size_t)C * N * 4, cb = (size_t)C * 4;
    if (!dA) return EFLA_ERR_NULL;
    if (!all_aligned16({dA, dD, ddt_bias, dh0, dh_L})) return EFLA_ERR_ALIGN;
    if (B == 0 || L == 0) {  // no tokens: the sums are zero and the state's adjoint passes through
        if (overlaps(dh0, hb, dh_L, hb) && dh0 != dh_L) return EFLA_ERR_ALIAS;
        bool ok = cudaMemsetAsync(dA, 0, pb, st) == cudaSuccess;
        if (dD) ok = ok && cudaMemsetAsync(dD, 0, cb, st) == cudaSuccess;
        if (ddt_bias) ok = ok && cudaMemsetAsync(ddt_bias, 0, cb, st) == cudaSuccess;
        if (dh0 && hb && dh0 != dh_L)
            ok = ok && (dh_L ? cudaMemcpyAsync(dh0, dh_L, hb, cudaMemcpyDeviceToDevice, st)
                             : cudaMemsetAsync(dh0, 0, hb, st)) == cudaSuccess;
        return ok ? EFLA_OK : EFLA_ERR_CUDA;
    }
    if (ldx < C || lddt < C || (z && ldz < C) || ldb < (long long)G * N || ldc < (long long)G * N) return EFLA_ERR_SHAPE;
    if ((double)B * L * std::max({ldx, lddt, z ? ldz : 0, ldb, ldc}) > (double)kMaxElems) return EFLA_ERR_SHAPE;
    const scan::Plan p = scan_plan(B, L, C, G, N, true);
    if (!scan_fits(p)) return EFLA_ERR_SHAPE;
    if (!dy || !x || !dt || !A || !Bm || !Cm || !dx || !ddt || !dB || !dC || (z && !dz)) return EFLA_ERR_NULL;
    if (!aligned_to(x, e) || !aligned_to(dt, e) || !aligned_to(Bm, e) || !aligned_to(Cm, e) || !aligned_to(z, e) ||
        !aligned_to(lengths, 4) || !all_aligned16({dy, A, D, dt_bias, h0, dx, ddt, dB, dC, dz, workspace}))
        return EFLA_ERR_ALIGN;
    const BwdSizes z4 = bwd_sizes(p, B, L, C, G, N);
    if (!workspace || workspace_bytes < z4.bytes()) return EFLA_ERR_WORKSPACE;
    const long long rows = (long long)B * L;
    const size_t yb = (size_t)rows * C * e, gb = (size_t)rows * G * N * e;
    const Buf in[] = {{x, extent(rows, ldx, C, e)}, {dt, extent(rows, lddt, C, e)}, {z, extent(rows, ldz, C, e)},
                      {Bm, extent(rows, ldb, (long long)G * N, e)}, {Cm, extent(rows, ldc, (long long)G * N, e)},
                      {A, pb}, {D, cb}, {dt_bias, cb}, {lengths, (size_t)B * 4}, {h0, hb}, {dy, yb}, {dh_L, hb}};
    const Buf out[] = {{dx, yb}, {ddt, yb}, {dA, pb}, {dB, gb}, {dC, gb}, {dD, cb}, {z ? dz : nullptr, yb},
                       {ddt_bias, cb}, {dh0, hb}, {workspace, z4.bytes()}};
    if (aliased(in, out)) return EFLA_ERR_ALIAS;
    scan::Args a{};
    a.x = x; a.dt = dt; a.z = z; a.Bm = Bm; a.Cm = Cm;
    a.ldx = ldx; a.lddt = lddt; a.ldz = ldz; a.ldb = ldb; a.ldc = ldc;
    a.A = A; a.D = D; a.dt_bias = dt_bias; a.h0 = h0; a.lengths = lengths; a.softplus = softplus;
    a.B = B; a.L = L; a.C = C; a.G = G; a.N = N; a.tpg = p.tpg; a.nseg = p.nseg; a.seg = p.seg;
    a.dy = dy; a.dh_L = dh_L; a.dx = dx; a.ddt = ddt; a.dz = dz; a.dh0 = dh0;
    float *ws = static_cast<float *>(workspace);
    a.ckpt = ws;
    ws += z4.ckpt;
    a.part_bc = ws;
    ws += z4.bc;
    carve_segments(a, ws, true);
    a.part = ws;
    return dtype == EFLA_F32 ? run_scan_bwd<float>(a, p, dB, dC, dA, dD, ddt_bias, st)
                             : run_scan_bwd<__nv_bfloat16>(a, p, dB, dC, dA, dD, ddt_bias, st);
}

efla_status_t efla_scan_step(const void *x, long long ldx, const void *dt, long long lddt, const float *A,
                             const void *Bm, long long ldb, const void *Cm, long long ldc, const float *D,
                             const void *z, long long ldz, const float *dt_bias, efla_dtype_t dtype, int softplus,
                             float *h, void *y, int B, int C, int G, int N, efla_stream_t stream) {
    NvtxRange nvtx_("efla_scan_step");
    efla_status_t s = check_scan(dtype, B, 1, C, G, N);
    if (s != EFLA_OK) return s;
    if (B > 65535) return EFLA_ERR_SHAPE;
    if (B == 0 || C == 0) return EFLA_OK;
    if (ldx < C || lddt < C || (z && ldz < C) || ldb < (long long)G * N || ldc < (long long)G * N) return EFLA_ERR_SHAPE;
    if ((double)B * std::max({ldx, lddt, z ? ldz : 0, ldb, ldc}) > (double)kMaxElems) return EFLA_ERR_SHAPE;
    if (!x || !dt || !A || !Bm || !Cm || !h || !y) return EFLA_ERR_NULL;
    const size_t e = esize(dtype);
    if (!aligned_to(x, e) || !aligned_to(dt, e) || !aligned_to(Bm, e) || !aligned_to(Cm, e) || !aligned_to(z, e) ||
        !all_aligned16({A, D, dt_bias, h, y}))
        return EFLA_ERR_ALIGN;
    const Buf in[] = {{x, extent(B, ldx, C, e)}, {dt, extent(B, lddt, C, e)}, {z, extent(B, ldz, C, e)},
                      {Bm, extent(B, ldb, (long long)G * N, e)}, {Cm, extent(B, ldc, (long long)G * N, e)},
                      {A, (size_t)C * N * 4}, {D, (size_t)C * 4}, {dt_bias, (size_t)C * 4}};
    const Buf out[] = {{h, (size_t)B * C * N * 4}, {y, (size_t)B * C * e}};
    if (aliased(in, out)) return EFLA_ERR_ALIAS;
    scan::Args a{};
    a.x = x; a.dt = dt; a.z = z; a.Bm = Bm; a.Cm = Cm;
    a.ldx = ldx; a.lddt = lddt; a.ldz = ldz; a.ldb = ldb; a.ldc = ldc;
    a.A = A; a.D = D; a.dt_bias = dt_bias; a.h_L = h; a.y = y; a.softplus = softplus;
    a.B = B; a.L = 1; a.C = C; a.G = G; a.N = N;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
#define EFLA_STEP(T)                                                \
    switch (N) {                                                    \
        case 8: return launch_scan_step<T, 8>(a, st);               \
        case 16: return launch_scan_step<T, 16>(a, st);             \
        case 32: return launch_scan_step<T, 32>(a, st);             \
        default: return launch_scan_step<T, 64>(a, st);             \
    }
    if (dtype == EFLA_F32) { EFLA_STEP(float) }
    EFLA_STEP(__nv_bfloat16)
#undef EFLA_STEP
}

}  // extern "C"
