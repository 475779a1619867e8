// C-ABI of the block-scaled e4m3 operators (included by int8mm_api.cu, whose
// helpers it uses): argument checks, layouts, tensor maps and launches.

namespace {

constexpr int kFp8RowsMaxM = 1024;  // rows the weight-streaming kernel takes (its workspace is sized for them)
constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxTopK = 16;

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

bool dtype_ok(int dtype) { return dtype == INT8MM_F16 || dtype == INT8MM_BF16; }

// Rows per tile of the weight-streaming kernel for M rows.
int fp8_rows_nt(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

struct Fp8Layout {
    size_t codes, scales, total;
};

Fp8Layout fp8_weight_layout(int K, int N) {
    Fp8Layout L{};
    size_t o = align_up((size_t)N * K, 256);
    L.scales = o;
    L.total = align_up(o + (size_t)cdiv(N, 128) * cdiv(K, 128) * 4, 256);
    return L;
}

// Rows of the scales of X in the workspace (a block's scales are contiguous):
// whole tiles of the tiled kernel, which reads the scales of rows past M too.
long long fp8_pitch(int M) { return ((long long)M + 255) / 256 * 256; }

struct Fp8WsLayout {
    size_t status, codes, scales, tickets, parts, total;
};

Fp8WsLayout fp8_ws_layout(int M, int K, int N) {
    Fp8WsLayout L{};
    size_t o = 256;
    L.codes = o;
    o = align_up(o + (size_t)M * K, 256);
    L.scales = o;
    o = align_up(o + (size_t)fp8_pitch(M) * cdiv(K, 128) * 4, 256);
    L.tickets = o;
    L.parts = o;
    if (M <= kFp8RowsMaxM) {
        const int nt = fp8_rows_nt(M);
        o = align_up(o + (size_t)cdiv(N, 128) * cdiv(M, nt) * 4, 256);
        L.parts = o;
        o = align_up(o + (size_t)2 * kFRMaxCtas * std::min(M, nt) * 128 * 4, 256);
    }
    L.total = o;
    return L;
}

struct MoeWsLayout {
    size_t status, logits, ids, wts, active, masks, tickets, xq, xs, hq, hs, parts, total;
    size_t t_gate, t_down;  // tickets of the two products, after the router's
};

// Chosen experts of T tokens: at most min(E, T * top_k).
int moe_max_active(int T, int E, int top_k) { return (int)std::min<long long>(E, (long long)T * top_k); }

MoeWsLayout moe_ws_layout(int T, int H, int I, int E, int top_k) {
    MoeWsLayout L{};
    const int A = moe_max_active(T, E, top_k);
    size_t o = 256;
    const auto take = [&o](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes, 256);
        return at;
    };
    L.logits = take((size_t)T * E * 8);
    L.ids = take((size_t)T * top_k * 4);
    L.wts = take((size_t)T * top_k * 4);
    L.active = take((size_t)(A + 1) * 4);
    L.masks = take((size_t)A * 8);
    L.tickets = take((size_t)(T + 1) * 4);
    L.t_gate = take((size_t)A * cdiv(I, 128) * 4);
    L.t_down = take((size_t)cdiv(H, 128) * 4);
    L.xq = take((size_t)T * H);
    L.xs = take((size_t)T * cdiv(H, 128) * 4);
    L.hq = take((size_t)A * T * I);
    L.hs = take((size_t)A * T * cdiv(I, 128) * 4);
    L.parts = take((size_t)4 * kFRMaxCtas * T * 2 * 128 * 4);
    L.total = o;
    return L;
}

bool moe_shape_ok(int T, int H, int I, int E, int top_k) {
    // (at most 256 experts of 2^20 units of 16 KB: units are counted in 32 bits)
    return T >= 1 && T <= kMoeMaxTokens && shape_ok(T, H, I) && I <= kMaxK && E >= 1 && E <= kMaxExperts &&
           top_k >= 1 && top_k <= kMoeMaxTopK && top_k <= E;
}

// 3-D tensor of `depth` row-major matrices of `outer` rows x `inner` bytes,
// with a 128-byte swizzled box of 128 x box_outer x 1.
bool make_map3(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t depth, uint32_t box_outer) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {inner, outer, depth};
    cuuint64_t strides[2] = {inner, inner * outer};
    cuuint32_t box[3] = {128, box_outer, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Y (M x N, 16 bits) in boxes of 32 rows x 32 columns with the 64-byte swizzle.
bool make_map_y(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t N, uint64_t M) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {N, M};
    cuuint64_t strides[1] = {N * 2};
    cuuint32_t box[2] = {32, 32};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Opt in to a kernel's shared memory once per device, and refuse a kernel
// whose launch holds fewer registers than its setmaxnreg split hands out.
template <auto Kern, int kMinRegs = 0>
cudaError_t fp8_opt_in(int dev, int smem) {
    static std::atomic<uint64_t> done{0};  // one bit per device (current_device admits fewer than 64)
    if ((done.load(std::memory_order_acquire) >> dev) & 1u) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && kMinRegs > 0) {
        cudaFuncAttributes a{};
        e = cudaFuncGetAttributes(&a, Kern);
        if (e == cudaSuccess && a.numRegs < kMinRegs) e = cudaErrorInvalidConfiguration;
    }
    if (e == cudaSuccess) done.fetch_or(1ull << dev, std::memory_order_release);
    return e;
}

cudaError_t launch_quant_fp8(const uint16_t* X, int dtype, int M, int K, uint8_t* codes, float* scales, long long sm,
                             long long sb, int sms, cudaStream_t s) {
    const int KB = cdiv(K, 128);
    const long long nblocks = (long long)M * KB;
    const long long per = (long long)(kQuantThreads / 8) * kQuantBlocks;
    const int grid = (int)std::max<long long>(1, std::min<long long>((nblocks + per - 1) / per, (long long)sms * 16));
    return dtype == INT8MM_F16
               ? launch(k_quant_fp8<F16>, dim3(grid), dim3(kQuantThreads), 0, s, true, X, nblocks, K, KB, codes, scales,
                        sm, sb)
               : launch(k_quant_fp8<BF16>, dim3(grid), dim3(kQuantThreads), 0, s, true, X, nblocks, K, KB, codes,
                        scales, sm, sb);
}

template <int kMode, int kNT, bool kFuse, typename T>
cudaError_t launch_rows(int dev, int grid, const CUtensorMap& tw, const CUtensorMap& tw2, const CUtensorMap& tx,
                        const CUtensorMap& tnext, const Fp8RowsParams& p, cudaStream_t s, bool pdl) {
    constexpr int smem = fr_smem_bytes<kMode, kNT>();
    static_assert(smem <= kMaxSmemOptin, "shared memory of one SM");
    cudaError_t e = fp8_opt_in<k_fp8_rows<kMode, kNT, kFuse, T>>(dev, smem);
    if (e != cudaSuccess) return e;
    return launch_ex(k_fp8_rows<kMode, kNT, kFuse, T>, dim3(grid), dim3(fr_threads<kNT>()), smem, s, pdl,
                     p.cut > 1 ? p.cut : 0, tw, tw2, tx, tnext, p);
}

template <int kBN, typename T>
cudaError_t launch_gemm_fp8(int dev, int grid, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& ty,
                            const Fp8GemmParams& p, cudaStream_t s, bool pdl) {
    cudaError_t e = fp8_opt_in<k_gemm_fp8_2sm<kBN, T>, kF8LaunchRegs>(dev, f8_smem_bytes(kBN));
    if (e != cudaSuccess) return e;
    return launch_ex(k_gemm_fp8_2sm<kBN, T>, dim3(grid), dim3(kF8Threads), f8_smem_bytes(kBN), s, pdl, 2, ta, tb, ty, p);
}

struct Fp8Opts {
    int path;
    cudaEvent_t ev0, ev1;
    uint64_t wait_ns;
    uint32_t test_flags;
};

bool fp8_opts(const int8mm_forward_opts* o, Fp8Opts* out) {
    *out = Fp8Opts{INT8MM_PATH_AUTO, nullptr, nullptr, kDefaultWaitNs, 0};
    if (!o) return true;
    if (o->acc_out) return false;  // there are no int32 sums
    out->path = o->path;
    out->ev0 = reinterpret_cast<cudaEvent_t>(o->main_start_event);
    out->ev1 = reinterpret_cast<cudaEvent_t>(o->main_stop_event);
    if (o->wait_limit_ns) out->wait_ns = o->wait_limit_ns;
    out->test_flags = o->test_flags;
    return (out->ev0 == nullptr) == (out->ev1 == nullptr);
}

// Into how many pieces the weight-streaming kernel cuts each of `tiles` tiles
// for a cluster of as many blocks (1: a tile per block), or 0 for equal runs
// of units that are joined through memory.  A tile has `units` units, at least
// `least` of them (they differ where the device decides on the experts).
// More tiles than SMs: runs.  Else the shortest by an estimate, whose figures
// are fits to the plain product at K = 512 .. 16384, N = 1024 .. 18432 with 8, 24,
// 48 and 100 rows; there its choice was within 4 % of the best one.  (It takes a
// stream for faster than one block's from HBM, 280 ns a unit, and runs for as many
// shares as there are SMs: see the down product's use of it.)  Runs against this choice:
// 8 rows, 4096 x 11008 13.7 -> 12.6 us (not cut), 8192 x 1024 11.4 -> 7.1 (8
// pieces), 1024 x 14336 8.4 -> 6.4 (not cut); 100 rows, 4096 x 11008 23.0 ->
// 18.5 (not cut), 11008 x 4096 24.0 -> 18.9 (4 pieces), but 16384 x 9728 stays
// with runs (41.6, not cut 54.3).
int fp8_cut(DeviceInfo* info, int tiles, int units, int least, int nt, int ctas) {
    if (tiles > ctas) return 0;
    // ns: a unit in one block; a join through memory, and more of it for each
    // block that shares the tile; a join in a cluster
    static constexpr struct {
        double unit, join, share, cluster;
    } kCost[4] = {{240, 2000, 200, 900}, {200, 2000, 200, 700}, {275, 4300, 370, 1900}, {370, 9000, 700, 2000}};
    const auto& k = kCost[nt == 16 ? 0 : nt == 32 ? 1 : nt == 64 ? 2 : 3];
    const double hbm = 2.5 * tiles * units;  // every unit from HBM
    const int most = std::min(8, ctas / tiles);
    double best = std::max(k.unit * tiles * units / ctas, hbm) + k.join + k.share * ctas / tiles;
    int cut = 0;
    for (int c = 1; c <= most && (c == 1 || 2 * c <= least); ++c) {
        const double t = std::max(k.unit * cdiv(units, c), hbm) + (c > 1 ? k.cluster : 0);
        if (t <= best && (c == 1 || c * tiles <= cluster_capacity(info, c) * c)) {
            best = t;
            cut = c;
        }
    }
    return cut;
}

// Whether the weight-streaming kernel takes a product of M rows: up to 128 rows
// each weight box is read once (100 x 11008 x 4096: 19 us against 46 us tiled);
// above, as long as its 128 x 128 tiles are one wave (512 x 4096 x 4096: 20.5
// against 22.8 us; 256 x 4096 x 11008, two waves: 33.4 against 23.3 us).
bool fp8_rows_path(int M, int N, int sms) {
    return M <= 128 || (M <= kFp8RowsMaxM && (long long)cdiv(M, 128) * cdiv(N, 128) <= sms);
}

}  // namespace

extern "C" {

int8mm_status int8mm_quantize_fp8(const uint16_t* X, int dtype, int M, int K, uint8_t* codes, float* scales,
                                  void* stream) {
    if (!X || !codes || !scales || !dtype_ok(dtype) || !shape_ok(M, K, 16)) return INT8MM_ERR_INVALID_ARGUMENT;
    if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return INT8MM_ERR_MISALIGNED;
    const size_t values = (size_t)M * K, blocks = (size_t)M * cdiv(K, 128);
    if (overlap(X, 2 * values, codes, values) || overlap(X, 2 * values, scales, 4 * blocks) ||
        overlap(codes, values, scales, 4 * blocks))
        return INT8MM_ERR_INVALID_ARGUMENT;
    int dev;
    DeviceInfo* info;
    int8mm_status st = current_device(&dev, &info);
    if (st != INT8MM_OK) return st;
    return cuda_status(launch_quant_fp8(X, dtype, M, K, codes, scales, cdiv(K, 128), 1, info->sm_count,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

size_t int8mm_fp8_weight_bytes(int K, int N) {
    if (!shape_ok(1, K, N)) return 0;
    return fp8_weight_layout(K, N).total;
}

int8mm_status int8mm_prepare_weight_fp8(const uint16_t* W, int dtype, int K, int N, void* buf, size_t buf_bytes,
                                        int8mm_fp8_weight* out, void* stream) {
    if (!W || !buf || !out || !dtype_ok(dtype) || !shape_ok(1, K, N)) return INT8MM_ERR_INVALID_ARGUMENT;
    if (!aligned(W, 16) || !aligned(buf, 256)) return INT8MM_ERR_MISALIGNED;
    const Fp8Layout L = fp8_weight_layout(K, N);
    if (buf_bytes < L.total) return INT8MM_ERR_WORKSPACE_TOO_SMALL;
    int dev;
    DeviceInfo* info;
    int8mm_status st = current_device(&dev, &info);
    if (st != INT8MM_OK) return st;
    uint8_t* b = static_cast<uint8_t*>(buf);
    int8mm_fp8_weight w{};
    w.K = K;
    w.N = N;
    w.codes = b;
    w.scales = reinterpret_cast<float*>(b + L.scales);
    const dim3 grid(cdiv(N, 128), cdiv(K, 128));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == INT8MM_F16
                              ? launch(k_quant_weight_fp8<F16>, grid, dim3(256), 0, s, false, W, K, N, w.codes, w.scales)
                              : launch(k_quant_weight_fp8<BF16>, grid, dim3(256), 0, s, false, W, K, N, w.codes, w.scales);
    if (e != cudaSuccess) return cuda_status(e);
    *out = w;
    return INT8MM_OK;
}

size_t int8mm_fp8_workspace_bytes(int M, int K, int N) {
    if (!shape_ok(M, K, N)) return 0;
    return fp8_ws_layout(M, K, N).total;
}

int8mm_status int8mm_forward_fp8(const uint16_t* X, int dtype, int M, const int8mm_fp8_weight* w, uint16_t* Y, void* ws,
                                 size_t ws_bytes, const int8mm_forward_opts* opts, void* stream) {
    if (!X || !w || !Y || !ws || !w->codes || !w->scales || !dtype_ok(dtype)) return INT8MM_ERR_INVALID_ARGUMENT;
    const int K = w->K, N = w->N;
    Fp8Opts o;
    if (!shape_ok(M, K, N) || !fp8_opts(opts, &o)) return INT8MM_ERR_INVALID_ARGUMENT;
    if (o.path != INT8MM_PATH_AUTO && o.path != INT8MM_PATH_GEMM && o.path != INT8MM_PATH_DECODE)
        return INT8MM_ERR_INVALID_ARGUMENT;
    if (o.path == INT8MM_PATH_DECODE && M > kFp8RowsMaxM) return INT8MM_ERR_INVALID_ARGUMENT;
    // tiles and 16 KB units are counted in 32 bits (units of at most 8 row blocks: a weight of 2 TB)
    if (M <= kFp8RowsMaxM && (long long)cdiv(N, 128) * cdiv(M, fp8_rows_nt(M)) * cdiv(K, 128) > (INT32_MAX >> 1))
        return INT8MM_ERR_INVALID_ARGUMENT;
    if ((long long)cdiv(N, 128) * cdiv(M, kF8BM) > (INT32_MAX >> 1)) return INT8MM_ERR_INVALID_ARGUMENT;
    if (!aligned(X, 16) || !aligned(Y, 16) || !aligned(ws, 256) || !aligned(w->codes, 16) || !aligned(w->scales, 4))
        return INT8MM_ERR_MISALIGNED;
    const Fp8WsLayout L = fp8_ws_layout(M, K, N);
    if (ws_bytes < L.total) return INT8MM_ERR_WORKSPACE_TOO_SMALL;
    // up to 16 rows are quantised by the blocks that multiply them, beside others' stores to Y
    if (overlap(X, (size_t)M * K * 2, Y, (size_t)M * N * 2)) return INT8MM_ERR_INVALID_ARGUMENT;
    int dev;
    DeviceInfo* info;
    int8mm_status st = current_device(&dev, &info);
    if (st != INT8MM_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* b = static_cast<uint8_t*>(ws);
    uint8_t* xq = b + L.codes;
    float* xs = reinterpret_cast<float*>(b + L.scales);
    const int KB = cdiv(K, 128), sms = std::min(info->sm_count, kFRMaxCtas);
    const bool f16 = dtype == INT8MM_F16, timed = o.ev0 != nullptr;
    const bool rows = o.path == INT8MM_PATH_DECODE || (o.path == INT8MM_PATH_AUTO && fp8_rows_path(M, N, sms));
    const int nt = fp8_rows_nt(M);
    // up to 16 rows each block quantises them again and a launch is saved (16 x 4096 x 4096: 8.0
    // us against 9.0); more keep the side warps too busy (32 x 4096 x 11008: 20.2 against 15.5)
    const bool fuse = rows && nt <= 16;
    cudaError_t e = cudaSuccess;
    if (!fuse) e = launch_quant_fp8(X, dtype, M, K, xq, xs, 1, fp8_pitch(M), info->sm_count, s);
    if (e != cudaSuccess) return cuda_status(e);
    CUtensorMap ta, tb;
    if (rows) {
        Fp8RowsParams p{};
        p.M = M;
        p.N = N;
        p.K = K;
        p.KB = KB;
        p.NB = cdiv(N, 128);
        p.MB = cdiv(M, nt);
        p.X = X;
        p.xs = xs;
        p.xs_pitch = fp8_pitch(M);
        p.ws = w->scales;
        p.Y = Y;
        p.parts = reinterpret_cast<float*>(b + L.parts);
        p.part_rows = std::min(M, nt);
        p.tickets = reinterpret_cast<unsigned*>(b + L.tickets);
        p.status = reinterpret_cast<int*>(b + L.status);
        p.wait_limit_ns = o.wait_ns;
        p.test_flags = o.test_flags;
        if (!make_map(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, w->codes, K, N, K, 128, 128)) return INT8MM_ERR_CUDA;
        tb = ta;  // unused when the codes are made in the kernel
        if (!fuse && !make_map(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, K, M, K, 128, (uint32_t)nt)) return INT8MM_ERR_CUDA;
        p.cut = fp8_cut(info, p.NB * p.MB, KB, KB, nt, sms);
        p.shares = FrShares(p.NB * p.MB, KB, sms, p.cut);
        const int grid = p.shares.count;
        if (timed) e = cudaEventRecord(o.ev0, s);
        if (e != cudaSuccess) return cuda_status(e);
        const bool pdl = !timed;
#define I8_ROWS(NT, FUSE)                                                                           \
    (f16 ? launch_rows<kRows, NT, FUSE, F16>(dev, grid, ta, ta, tb, ta, p, s, pdl)                  \
         : launch_rows<kRows, NT, FUSE, BF16>(dev, grid, ta, ta, tb, ta, p, s, pdl))
        e = nt == 16 ? I8_ROWS(16, true) : nt == 32 ? I8_ROWS(32, false) : nt == 64 ? I8_ROWS(64, false) : I8_ROWS(128, false);
#undef I8_ROWS
    } else {
        constexpr int bn = 256;
        CUtensorMap ty;
        if (!make_map(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, K, M, K, 128, 128) ||
            !make_map(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, w->codes, K, N, K, 128, bn / 2) ||
            !make_map_y(&ty, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, Y, N, M))
            return INT8MM_ERR_CUDA;
        Fp8GemmParams p{};
        p.M = M;
        p.N = N;
        p.KB = KB;
        p.num_m_blocks = cdiv(M, kF8BM);
        p.num_n_blocks = cdiv(N, bn);
        p.num_tiles = p.num_m_blocks * p.num_n_blocks;
        // the largest group of row blocks whose codes fit in 48 MB of L2, at least 8
        const int fit = (int)std::min<uint64_t>(1u << 20, (48ull << 20) / ((uint64_t)kF8BM * (uint64_t)K));
        p.group_m = std::min(std::max(8, fit), p.num_m_blocks);
        p.xs = xs;
        p.xs_pitch = fp8_pitch(M);
        p.ws = w->scales;
        p.status = reinterpret_cast<int*>(b + L.status);
        p.wait_limit_ns = o.wait_ns;
        p.test_flags = o.test_flags;
        const int grid = 2 * std::min(p.num_tiles, info->sm_count / 2);
        if (timed) e = cudaEventRecord(o.ev0, s);
        if (e != cudaSuccess) return cuda_status(e);
        e = f16 ? launch_gemm_fp8<bn, F16>(dev, grid, ta, tb, ty, p, s, !timed)
                : launch_gemm_fp8<bn, BF16>(dev, grid, ta, tb, ty, p, s, !timed);
    }
    if (e == cudaSuccess && timed) e = cudaEventRecord(o.ev1, s);
    return cuda_status(e);
}

size_t int8mm_moe_workspace_bytes(int T, int H, int I, int E, int top_k) {
    if (!moe_shape_ok(T, H, I, E, top_k)) return 0;
    return moe_ws_layout(T, H, I, E, top_k).total;
}

int8mm_status int8mm_forward_moe_fp8(const uint16_t* X, int dtype, int T, const int8mm_moe_weight* w, int top_k,
                                     int renormalize, uint16_t* Y, int32_t* topk_ids, float* topk_weights, void* ws,
                                     size_t ws_bytes, const int8mm_forward_opts* opts, void* stream) {
    if (!X || !w || !Y || !ws || !dtype_ok(dtype) || !w->router || !w->gate_codes || !w->gate_scales || !w->up_codes ||
        !w->up_scales || !w->down_codes || !w->down_scales)
        return INT8MM_ERR_INVALID_ARGUMENT;
    const int H = w->H, I = w->I, E = w->E;
    Fp8Opts o;
    if (!moe_shape_ok(T, H, I, E, top_k) || !fp8_opts(opts, &o) || o.path != INT8MM_PATH_AUTO || o.ev0)
        return INT8MM_ERR_INVALID_ARGUMENT;
    if (!aligned(X, 16) || !aligned(Y, 16) || !aligned(ws, 256) || !aligned(w->router, 16) ||
        !aligned(w->gate_codes, 16) || !aligned(w->up_codes, 16) || !aligned(w->down_codes, 16) ||
        !aligned(w->gate_scales, 4) || !aligned(w->up_scales, 4) || !aligned(w->down_scales, 4) ||
        !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
        return INT8MM_ERR_MISALIGNED;
    const MoeWsLayout L = moe_ws_layout(T, H, I, E, top_k);
    if (ws_bytes < L.total) return INT8MM_ERR_WORKSPACE_TOO_SMALL;
    // What the kernels write lies on nothing else (the lists in the workspace and topk_ids are
    // indexes that later blocks use, and routing is stored while other blocks still read X); only
    // Y, which is written last, may lie on X.
    const size_t values = (size_t)E * H * I, block_scales = (size_t)E * cdiv(H, 128) * cdiv(I, 128) * 4;
    const size_t routed = (size_t)T * top_k * 4, tokens = (size_t)T * H * 2;
    const struct {
        const void* at;
        size_t bytes;
    } parts[] = {{ws, L.total}, {topk_ids, topk_ids ? routed : 0}, {topk_weights, topk_weights ? routed : 0}, {Y, tokens},
                 {X, tokens}, {w->router, (size_t)E * H * 2}, {w->gate_codes, values}, {w->up_codes, values},
                 {w->down_codes, values}, {w->gate_scales, block_scales}, {w->up_scales, block_scales},
                 {w->down_scales, block_scales}};
    constexpr int kWritten = 4, kY = 3, kX = 4;
    for (int i = 0; i < kWritten; ++i)
        for (int j = i + 1; parts[i].bytes && j < (int)(sizeof(parts) / sizeof(parts[0])); ++j)
            if (!(i == kY && j == kX) && parts[j].bytes && overlap(parts[i].at, parts[i].bytes, parts[j].at, parts[j].bytes))
                return INT8MM_ERR_INVALID_ARGUMENT;
    int dev;
    DeviceInfo* info;
    int8mm_status st = current_device(&dev, &info);
    if (st != INT8MM_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* b = static_cast<uint8_t*>(ws);
    const int A = moe_max_active(T, E, top_k), HB = cdiv(H, 128), IB = cdiv(I, 128), nt = fp8_rows_nt(T);
    const int ctas = std::min(info->sm_count, kFRMaxCtas);
    const bool f16 = dtype == INT8MM_F16;
    int32_t* ids = topk_ids ? topk_ids : reinterpret_cast<int32_t*>(b + L.ids);
    float* wts = topk_weights ? topk_weights : reinterpret_cast<float*>(b + L.wts);

    CUtensorMap tg, tu, td, tx, th;
    if (!make_map3(&tg, w->gate_codes, H, I, E, 128) || !make_map3(&tu, w->up_codes, H, I, E, 128) ||
        !make_map3(&td, w->down_codes, I, H, E, 128) ||
        !make_map(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, b + L.xq, H, T, H, 128, (uint32_t)nt) ||
        !make_map3(&th, b + L.hq, I, T, A, (uint32_t)nt))
        return INT8MM_ERR_CUDA;

    RouteParams r{};
    r.X = X;
    r.R = w->router;
    r.T = T;
    r.H = H;
    r.E = E;
    r.top_k = top_k;
    r.renorm = renormalize != 0;
    const int tt = T == 1 ? 1 : 4;
    r.log_blocks = cdiv(E, kRouteExperts) * cdiv(T, tt);
    r.logits = reinterpret_cast<double*>(b + L.logits);
    r.ids = ids;
    r.wts = wts;
    r.active = reinterpret_cast<int32_t*>(b + L.active);
    r.masks = reinterpret_cast<unsigned long long*>(b + L.masks);
    r.tickets = reinterpret_cast<unsigned*>(b + L.tickets);
    r.xq = b + L.xq;
    r.xs = reinterpret_cast<float*>(b + L.xs);
    const dim3 rgrid(r.log_blocks + cdiv((long long)T * HB, kRouteThreads / 8));
    cudaError_t e;
#define I8_ROUTE(TT) \
    (f16 ? launch(k_moe_route<TT, F16>, rgrid, dim3(kRouteThreads), 0, s, true, r) \
         : launch(k_moe_route<TT, BF16>, rgrid, dim3(kRouteThreads), 0, s, true, r))
    e = tt == 1 ? I8_ROUTE(1) : I8_ROUTE(4);
#undef I8_ROUTE
    if (e != cudaSuccess) return cuda_status(e);

    Fp8RowsParams p{};
    p.M = T;
    p.MB = 1;
    p.active = r.active;
    p.max_active = A;
    p.masks = r.masks;
    p.ids = ids;
    p.wts = wts;
    p.top_k = top_k;
    p.hq = b + L.hq;
    p.hs = reinterpret_cast<float*>(b + L.hs);
    p.parts = reinterpret_cast<float*>(b + L.parts);
    p.part_rows = T;
    p.status = reinterpret_cast<int*>(b + L.status);
    p.wait_limit_ns = o.wait_ns;
    p.test_flags = o.test_flags;
    Fp8RowsParams g = p;
    g.N = I;
    g.K = H;
    g.KB = HB;
    g.NB = IB;
    g.xs = r.xs;
    g.xs_pitch = T;
    g.ws = w->gate_scales;
    g.ws2 = w->up_scales;
    g.tickets = reinterpret_cast<unsigned*>(b + L.t_gate);
    // (how many experts the tokens reach is known on the device only: blocks past the shares leave)
    const int ggrid = std::min(ctas, std::max(A * IB, A * IB * HB / kFRMinUnits));
    // (the chosen experts are at least top_k)
    g.next_cut = fp8_cut(info, HB, A * IB, top_k * IB, nt, ctas);
    // Clusters that leave SMs idle lose against runs where much weight is read (us a layer, clusters
    // against runs: 16 tokens, 8 of 64 experts, 2048 x 1408, 104.2 / 99.6; 8 of 128, 2048 x 768,
    // 88.2 / 84.2; 32 tokens 121.9 / 114.1 and 117.6 / 110.4).  The rule does not look at how much
    // that is, and smaller layers lose by it (16 tokens, 2 of 8, 256 x 512, 18.3 / 21.0; 512 x 1408,
    // 20.4 / 27.4; 1024 x 2816, 33.9 / 38.0; 8 of 64, 512 x 256, 26.0 / 32.6; one token, 2 of 8,
    // 4096 x 272, 20.9 / 23.3).
    if (nt <= 32 && 5 * g.next_cut * HB < 4 * ctas) g.next_cut = 0;
    g.next_grid = g.next_cut ? g.next_cut * HB : std::min(ctas, std::max(HB, A * IB * HB / kFRMinUnits));
    e = nt == 16   ? launch_rows<kGateUp, 16, false, F16>(dev, ggrid, tg, tu, tx, td, g, s, true)
        : nt == 32 ? launch_rows<kGateUp, 32, false, F16>(dev, ggrid, tg, tu, tx, td, g, s, true)
                   : launch_rows<kGateUp, 64, false, F16>(dev, ggrid, tg, tu, tx, td, g, s, true);
    if (e != cudaSuccess) return cuda_status(e);
    Fp8RowsParams d = p;
    d.N = H;
    d.K = I;
    d.KB = IB;
    d.NB = HB;
    d.xs = p.hs;
    d.xs_pitch = T;
    d.ws = w->down_scales;
    d.Y = Y;
    d.test_flags = 0;
    d.tickets = reinterpret_cast<unsigned*>(b + L.t_down);
    d.cut = g.next_cut;
    const int dgrid = g.next_grid;
#define I8_DOWN(NT)                                                                        \
    (f16 ? launch_rows<kDown, NT, false, F16>(dev, dgrid, td, td, th, td, d, s, true)          \
         : launch_rows<kDown, NT, false, BF16>(dev, dgrid, td, td, th, td, d, s, true))
    e = nt == 16 ? I8_DOWN(16) : nt == 32 ? I8_DOWN(32) : I8_DOWN(64);
#undef I8_DOWN
    return cuda_status(e);
}

}  // extern "C"
