// C entry points of the row-softmax operators: cross attention and softmax
// cross entropy.  Host code (but for the error word): argument checks, the choice
// between the tensor-core and the CUDA-core kernels, the plan of splits and
// pieces, the layout of the caller's workspace, and the launches.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "fs_ops.cuh"

namespace {

__device__ int g_ops_err;    // error bits of the handle-less calls on this device
__device__ int g_ops_taken;  // those that the fs_check under way has taken

// In one step, so that a bit that another stream's kernel raises meanwhile is taken now or stays for the next check.
__global__ void take_errors_kernel() { g_ops_taken = atomicExch(&g_ops_err, 0); }

constexpr int kMaxDevices = 64;
constexpr unsigned long long kTimeoutNs = 2000000000ull;

fs_status reject(fs_status st, const char *fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    fs::set_thread_error(buf);
    return st;
}

#define OPS_LAUNCH(call, kernels)                                                                \
    do {                                                                                         \
        cudaError_t e_ = (call);                                                                 \
        if (e_ != cudaSuccess) return reject(FS_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_)); \
        fs::count_launches(kernels);                                                             \
    } while (0)

struct Device {
    bool ready = false;
    int sms = 0, pairs = 0;  // SMs; CTA pairs of the cross-entropy kernel that run at once
    int *err = nullptr;
};

// The current device's properties and error word, looked up once per device.
fs_status current_device(Device *out) {
    static std::mutex mu;
    static Device known[kMaxDevices];
    int dev = 0, major = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return reject(FS_ERR_CUDA, "no CUDA device: %s", cudaGetErrorString(e));
    if (dev >= kMaxDevices) return reject(FS_ERR_UNSUPPORTED, "device index beyond 63");
    std::lock_guard<std::mutex> lock(mu);
    Device &d = known[dev];
    if (!d.ready) {
        void *addr = nullptr;
        e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        if (e == cudaSuccess && major != 10) return reject(FS_ERR_UNSUPPORTED, "this library is built for sm_100a");
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaGetSymbolAddress(&addr, g_ops_err);
        if (e == cudaSuccess) e = fs::xent_tc_pairs(&d.pairs);
        if (e != cudaSuccess) return reject(FS_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
        d.err = static_cast<int *>(addr);
        d.ready = true;
    }
    *out = d;
    return FS_OK;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
int up(int a, int b) { return (a + b - 1) / b; }

// Whether a [batch][token][head][w] tensor with these strides holds every element at its own address.
bool distinct(const fs_view &s, int batch, int tokens, int heads, int w) {
    struct Dim {
        long long stride, size;
    } dims[3] = {{s.batch, batch}, {s.token, tokens}, {s.head, heads}};
    std::sort(dims, dims + 3, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
    long long extent = w;  // elements spanned so far
    for (const Dim &x : dims) {
        if (x.size <= 1) continue;
        if (x.stride < extent) return false;
        extent = x.stride * (x.size - 1) + extent;
    }
    return true;
}
bool nonneg(const fs_view &s) { return s.batch >= 0 && s.token >= 0 && s.head >= 0; }

bool scale_ok(float s) { return s > 0.f && std::isfinite(s * fs::kLog2e); }

// ------------------------------------------------------------------ cross attention
fs_status check_attn(const fs_attn_desc *D, bool grad) {
    if (!D) return reject(FS_ERR_INVALID_ARG, "null descriptor");
    if (D->batch < 0 || D->n < 0 || D->m < 0) return reject(FS_ERR_INVALID_ARG, "batch, n and m must be >= 0");
    if (D->heads < 1 || D->kv_heads < 1 || D->heads % D->kv_heads)
        return reject(FS_ERR_INVALID_ARG, "heads must be a positive multiple of kv_heads");
    if (D->d < 1 || D->dv < 1 || D->d > 256 || D->dv > 256)
        return reject(FS_ERR_INVALID_ARG, "d and dv must be 1 to 256");
    if (D->dtype != FS_F32 && D->dtype != FS_BF16) return reject(FS_ERR_INVALID_ARG, "unknown dtype");
    if (!scale_ok(D->scale)) return reject(FS_ERR_INVALID_ARG, "scale must be > 0, and finite times log2(e)");
    if (!nonneg(D->q) || !nonneg(D->k) || !nonneg(D->v) || !nonneg(D->out) ||
        (grad && (!nonneg(D->dout) || !nonneg(D->dq) || !nonneg(D->dk) || !nonneg(D->dvw))))
        return reject(FS_ERR_INVALID_ARG, "strides must be >= 0");
    if ((long long)D->batch * D->heads > 65535)
        return reject(FS_ERR_UNSUPPORTED, "batch * heads exceeds 65535");
    if ((long long)D->n * D->heads >= 1ll << 27 || D->m >= 1 << 30)
        return reject(FS_ERR_UNSUPPORTED, "n * heads is 2^27 or more, or m 2^30 or more");
    const bool ok = grad ? distinct(D->dq, D->batch, D->n, D->heads, D->d) &&
                               distinct(D->dk, D->batch, D->m, D->kv_heads, D->d) &&
                               distinct(D->dvw, D->batch, D->m, D->kv_heads, D->dv)
                         : distinct(D->out, D->batch, D->n, D->heads, D->dv);
    if (!ok) return reject(FS_ERR_INVALID_ARG, "an output's strides make elements overlap");
    return FS_OK;
}

struct AttnPlan {
    int unit_rows = 0, blocks = 0, main_units = 0, tail_units = 0, splits = 1, split_keys = 0;  // as in AttnParams
    int key_parts = 1, row_parts = 1;
    size_t part_dk = 0, part_dv = 0, part_dq = 0;
    size_t part_ml = 0, part_o = 0, dot = 0, lse2 = 0, top = 0, total = 0;  // workspace offsets, and its size
};

// kind: the kernels that take the call.
enum AttnKind { kSimt = 0, kTensor = 1, kToken = 2 };
AttnPlan plan_attn(const fs_attn_desc &D, bool grad, AttnKind kind, bool ragged, const Device &dev) {
    const bool tc = kind == kTensor;
    AttnPlan L;
    const size_t rows = (size_t)D.n * (D.heads / D.kv_heads), heads = (size_t)D.batch * D.kv_heads;
    if (grad) {
        L.lse2 = align256((size_t)D.batch * D.heads * D.n * sizeof(float));
        L.top = 2 * L.lse2;
        L.total = L.top + align256(D.batch * sizeof(float));
        const int group = D.heads / D.kv_heads, wide = std::max(D.d, D.dv);
        if (rows == 0 || heads == 0 || D.m == 0) return L;
        if (!tc && fs::xattn_simt_rows(D.m + D.n * group, (int)heads, dev.sms) != 16) return L;
        // Where some CTAs would stream for longer than an even share of all tiles takes the CTAs that run at once (tensor
        // cores: one an SM; CUDA cores, blocks of 16: two, or four up to width 64, where more of them hide each other's
        // waits), their tiles are split to about that share, four a part at least (CUDA cores: three).  A tile of the
        // pass that keeps keys takes 1.25 of the other's: tensor cores 0.85 us at width 128, CUDA cores 3 us at width 64.
        // It has to save more than the joining pass costs, and the sums written and read back at 4 TB/s.  Tensor
        // cores, 2000 queries of 8 heads on one key head, 64 keys of 128: 232 us whole, 43 split; 1000 x 1000, 4 heads:
        // 21 whole, 24 split.  CUDA cores, fp32, 2 x 200 x 300, 4 on 2 heads of 40: 75 whole, 45 split; 4 heads: 44
        // whole, 47 split.  (Shares take the work as divisible: that whole waves may end with few CTAs is not counted.)
        const size_t side = tc ? 128 : 16;
        const double slots = dev.sms * (tc ? 1.0 : wide <= 64 ? 4.0 : 2.0);
        const size_t key_blocks = (D.m + side - 1) / side, row_blocks = (rows + side - 1) / side;
        const int key_tiles = tc ? group * up(D.n, 64) : up((int)rows, 32), row_tiles = up(D.m, tc ? 64 : 32);
        const double least = tc ? 4.0 : 3.0, join_us = tc ? 8.5 : 15.0;
        const double tile_us = tc ? 0.85 : 3.0 * std::max(64, wide) / 64;
        const double each = (key_blocks * 1.25 * key_tiles + row_blocks * (double)row_tiles) * heads / slots;
        const int kp = (int)std::min({std::max(1.0, key_tiles * 1.25 / each), std::max(1.0, key_tiles / least), 64.0});
        const int rp = (int)std::min({std::max(1.0, row_tiles / each), std::max(1.0, row_tiles / least), 64.0});
        const size_t dk = kp > 1 ? kp * heads * key_blocks * side * D.d * sizeof(float) : 0;
        const size_t dv = kp > 1 ? kp * heads * key_blocks * side * D.dv * sizeof(float) : 0;
        const size_t dq = rp > 1 ? rp * heads * row_blocks * side * D.d * sizeof(float) : 0;
        const double before = std::max({key_tiles * 1.25, (double)row_tiles, each});
        const double after = std::max({key_tiles * 1.25 / kp, (double)row_tiles / rp, each}) +
                             (join_us + 2.0 * (dk + dv + dq) / 4e6) / tile_us;
        if ((kp > 1 || rp > 1) && after < before) {
            L.key_parts = kp;
            L.row_parts = rp;
            L.part_dk = L.total;
            L.part_dv = L.part_dk + align256(dk);
            L.part_dq = L.part_dv + align256(dv);
            L.total = L.part_dq + align256(dq);
        }
        return L;
    }
    if (rows == 0 || heads == 0) return L;
    // Rows of a unit (tensor cores: 128, or 256 in two blocks that share every tile), and which units are split over
    // their keys: what costs least, in tiles of 128 keys.  All of it was measured at width 128 on the tensor cores and
    // serves the other widths and kernels too.  A CTA takes its tiles (two blocks: 1.28 times as long each,
    // 2.3 us against 1.8 at width 128) and 1.5 tiles' time to start and end; waves of CTAs, one an SM (CUDA cores:
    // two).  With lengths, the longest problems come first and short ones fill in, so that the waves need not be whole,
    // and parts of unequal problems cost more (32 requests of up to 4096 keys: 66 us in one part, 89 in two; 8: 52 in
    // one, 33 in two, 30 in three, 37 in four; 32 of 4096 each: 100 whole, 104 with the last wave in four parts).
    // Either every unit is split, or only those behind the last full wave, so that they fill the SMs too; the joining
    // pass costs a launch, and the parts' sums written and read back (4 TB/s, 1.8 us a tile).
    const int slots = tc ? dev.sms : 2 * dev.sms;
    const int side = tc               ? 128
                     : kind == kToken ? (rows <= 2 ? (int)rows : 4)
                                      : fs::xattn_simt_rows(D.n * (D.heads / D.kv_heads), (int)heads, dev.sms);
    const int tile = 128, tiles = up(std::max(D.m, 1), tile);
    double best = 1e300;
    for (int two = 0; two < (tc && rows > 128 ? 2 : 1); ++two) {
        const int unit = side << two;
        const long long units = (long long)((rows + unit - 1) / unit * heads), rest = units % slots;
        const double per = two ? 1.28 : 1.0;
        auto consider = [&](long long tail, int s) {
            const int t = up(tiles, s), parts = up(tiles, t);
            const double live = (double)rows * heads / units;  // rows of a unit
            const double join = 2.0 + 0.02 * parts + tail * live * parts * D.dv * 8.0 / 4e6 / 1.8;
            const double n = (double)(tail * parts) / slots, ends = parts == 1 ? 1.5 : ragged ? 3.0 : 2.5;
            const double waves = ragged && n > 1.0 ? n + 0.1 : std::ceil(n);
            const double cost = (double)((units - tail) / slots) * (tiles * per + 1.5) + waves * (t * per + ends) +
                                (parts > 1 ? join : 0.0);
            if (cost < best - 1e-9) {
                best = cost;
                L.unit_rows = unit;
                L.blocks = (int)((rows + unit - 1) / unit);
                L.splits = parts;
                L.split_keys = t * tile;
                L.tail_units = parts > 1 ? (int)tail : 0;
                L.main_units = (int)(units - L.tail_units);
            }
        };
        // (numbers of parts that give the same tiles a part are one choice)
        for (int s = 1; s <= std::min(tiles, fs::kAttnParts) && (s == 1 || units < 3ll * slots); ++s)
            if (s == 1 || up(tiles, s) != up(tiles, s - 1)) consider(units, s);
        if (!ragged && units > slots && rest)
            for (int s = 2; s <= std::min(tiles, 16); ++s)
                if (up(tiles, s) != up(tiles, s - 1)) consider(rest, s);
    }
    if (L.splits > 1) {
        const size_t parts = (size_t)L.splits * L.tail_units * L.unit_rows;
        L.part_o = align256(parts * sizeof(fs::AttnPart));
        L.total = L.part_o + align256(parts * D.dv * sizeof(float));
    }
    return L;
}
size_t attn_workspace(const fs_attn_desc &D, bool grad, const Device &dev) {
    size_t most = 0;  // over the kernels and the lengths that a call may bring
    for (int k = 0; k < 6; ++k)
        if (k / 2 != kTensor || D.dtype == FS_BF16)
            most = std::max(most, plan_attn(D, grad, (AttnKind)(k / 2), k & 1, dev).total);
    return most;
}

// Whether the tensor-core kernels take the call: bf16, widths up to 128 and multiples of 8, keys to load, and
// bases and strides that 16-byte loads and TMA boxes can start on.
bool attn_tc_operands(const fs_attn_desc &D, const void *q, const void *k, const void *v) {
    return D.dtype == FS_BF16 && D.d <= 128 && D.dv <= 128 && D.d % 8 == 0 && D.dv % 8 == 0 && D.m > 0 &&
           fs::attn_tc_view(q, D.q, D.n, D.heads, D.batch, false) &&
           fs::attn_tc_view(k, D.k, D.m, D.kv_heads, D.batch, true) &&
           fs::attn_tc_view(v, D.v, D.m, D.kv_heads, D.batch, true);
}
bool attn_tc(const fs_attn_desc &D, const void *q, const void *k, const void *v, const void *out) {
    return attn_tc_operands(D, q, k, v) && fs::attn_tc_view(out, D.out, D.n, D.heads, D.batch, false);
}
bool attn_grad_tc(const fs_attn_desc &D, const void *q, const void *k, const void *v, const void *dout, const void *dq,
                  const void *dk, const void *dv) {
    return D.n > 0 && attn_tc_operands(D, q, k, v) && fs::attn_tc_view(q, D.q, D.n, D.heads, D.batch, true) &&
           fs::attn_tc_view(dout, D.dout, D.n, D.heads, D.batch, true) &&
           fs::attn_tc_view(dq, D.dq, D.n, D.heads, D.batch, false) &&
           fs::attn_tc_view(dk, D.dk, D.m, D.kv_heads, D.batch, false) &&
           fs::attn_tc_view(dv, D.dvw, D.m, D.kv_heads, D.batch, false);
}

fs::AttnParams attn_params(const fs_attn_desc &D, const AttnPlan &L, const Device &dev, void *ws) {
    fs::AttnParams p{};
    p.batch = D.batch;
    p.n = D.n;
    p.m = D.m;
    p.heads = D.heads;
    p.kv_heads = D.kv_heads;
    p.group = D.heads / D.kv_heads;
    int log = 0;
    while (1 << log < p.group) ++log;
    p.group_mul = (unsigned)(((1ull << (31 + log)) + p.group - 1) / p.group);
    p.group_shift = (unsigned)std::max(0, log - 1);
    p.d = D.d;
    p.dv = D.dv;
    p.scale = D.scale;
    p.scale2 = (float)((double)D.scale * fs::kLog2ed);
    p.qs = D.q;
    p.ks = D.k;
    p.vs = D.v;
    p.os = D.out;
    p.dos = D.dout;
    p.dqs = D.dq;
    p.dks = D.dk;
    p.dvs = D.dvw;
    p.unit_rows = L.unit_rows;
    p.blocks = L.blocks;
    p.main_units = L.main_units;
    p.tail_units = L.tail_units;
    p.splits = L.splits;
    p.split_keys = L.split_keys;
    char *w = static_cast<char *>(ws);
    p.key_parts = L.key_parts;
    p.row_parts = L.row_parts;
    p.part_dk = reinterpret_cast<float *>(w + L.part_dk);
    p.part_dv = reinterpret_cast<float *>(w + L.part_dv);
    p.part_dq = reinterpret_cast<float *>(w + L.part_dq);
    p.part_ml = reinterpret_cast<fs::AttnPart *>(w + L.part_ml);
    p.part_o = reinterpret_cast<float *>(w + L.part_o);
    p.dot = reinterpret_cast<float *>(w + L.dot);
    p.lse2 = reinterpret_cast<float *>(w + L.lse2);
    p.top = reinterpret_cast<float *>(w + L.top);
    p.timeout_ns = kTimeoutNs;
    p.err = dev.err;
    return p;
}

fs_status check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return FS_OK;
    if (!ws || have < need)
        return reject(FS_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", ws ? have : (size_t)0, need);
    if (reinterpret_cast<uintptr_t>(ws) & 255) return reject(FS_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
    return FS_OK;
}

// ------------------------------------------------------------------ cross entropy
fs_status check_xent(const fs_xent_desc *D, bool grad) {
    if (!D) return reject(FS_ERR_INVALID_ARG, "null descriptor");
    if (D->n < 0 || D->v < 1 || D->d < 1) return reject(FS_ERR_INVALID_ARG, "n must be >= 0, v and d >= 1");
    if (D->dtype != FS_F32 && D->dtype != FS_BF16) return reject(FS_ERR_INVALID_ARG, "unknown dtype");
    if (!scale_ok(D->scale)) return reject(FS_ERR_INVALID_ARG, "scale must be > 0, and finite times log2(e)");
    if (D->ldx < 0 || D->ldw < 0) return reject(FS_ERR_INVALID_ARG, "row strides must be >= 0");
    if (grad && ((D->n > 1 && D->lddx < D->d) || (D->v > 1 && D->lddw < D->d)))
        return reject(FS_ERR_INVALID_ARG, "an output's row stride is below d");
    if (D->v > 1 << 22 || D->d > 65536 || D->n > 1 << 24)
        return reject(FS_ERR_UNSUPPORTED, "v over 2^22, d over 65536 or n over 2^24");
    return FS_OK;
}

struct XentPlan {
    int planes = 1;            // bf16 planes of the products' operands
    bool pack_x = false, pack_w = false;  // copied into planes first (w piece by piece)
    int dp = 0;                // a plane's width
    int tiles = 0;             // column tiles of the forward
    int piece = 0, parts = 1;  // classes of a piece; parts of it in the dx product
    bool direct = false;       // one product is all of dx: written at once
    long long ld_dl = 0, ld_acc = 0;
    size_t px = 0, pw = 0, part = 0, hit = 0, dl = 0, acc = 0, total = 0;  // workspace offsets, and its size
};

XentPlan plan_xent(const fs_xent_desc &D, const void *x, const void *w, bool grad, const Device &dev) {
    XentPlan L;
    const bool f32 = D.dtype == FS_F32;
    const size_t n = (size_t)std::max(D.n, 1), room = (size_t)256 << 20;
    L.planes = f32 ? 3 : 1;
    // x is read again by every column tile: rows that do not start on 128 bytes take two lines of L2 a box row, and
    // are copied where there are enough tiles to repay it (1021 x 50021 x 1000: forward 89 us as they lie, 79 copied,
    // copy included; 512 x 16384 x 520: 19 against 21; w is read once a band of row tiles, and its copy does not pay).
    const bool lines = D.ldx % 64 == 0 && reinterpret_cast<uintptr_t>(x) % 128 == 0;
    L.pack_x = f32 || !fs::xent_tc_rows(x, D.ldx, D.n) || (!lines && (long long)D.n * D.v >= 1ll << 25);
    L.pack_w = f32 || !fs::xent_tc_rows(w, D.ldw, D.v);
    L.dp = up(D.d, 64) * 64;
    // Pieces of the classes whose logit gradients, and whose copies of w, stay within 256 MiB each.
    size_t fit = (size_t)up(D.v, 256) * 256;
    if (grad) fit = std::min(fit, room / (n * L.planes * 2) / 256 * 256);
    if (L.pack_w) fit = std::min(fit, room / ((size_t)L.dp * L.planes * 2) / 256 * 256);
    if (grad && f32) fit = std::min(fit, (size_t)8 * fs::kXentF32Terms);  // at most 8 parts of it in the dx product
    L.piece = (int)std::max<size_t>(256, fit);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += align256(bytes);
        return o;
    };
    if (L.pack_x) L.px = take(n * L.planes * L.dp * 2);
    if (L.pack_w) L.pw = take((size_t)std::min(L.piece, D.v) * L.planes * L.dp * 2);
    if (!grad) {
        L.tiles = up(D.v, fs::kXentCols);
        L.part = take((size_t)L.tiles * n * sizeof(float2));
        L.hit = take(n * sizeof(float));
    } else {
        L.ld_dl = L.piece;
        L.ld_acc = (D.d + 7) / 8 * 8;
        // dx: where the product's tiles are fewer than what runs at once, its sum over the classes is split.
        const long long tiles = (long long)up((int)n, 256) * up(D.d, 256);
        L.parts = (int)std::max(1ll, std::min<long long>(std::min(32ll, dev.pairs / tiles), L.piece / 512));
        if (f32) L.parts = std::max(L.parts, up(L.piece, fs::kXentF32Terms));
        L.direct = L.piece >= D.v && L.parts == 1;
        L.dl = take(n * L.planes * L.ld_dl * 2);
        if (!L.direct) L.acc = take((size_t)L.parts * n * L.ld_acc * sizeof(float));
    }
    L.total = at;
    return L;
}

fs::XentParams xent_params(const fs_xent_desc &D, const XentPlan &L, const Device &dev, void *ws, const void *x) {
    fs::XentParams p{};
    char *base = static_cast<char *>(ws);
    p.n = p.n_all = D.n;
    p.v = D.v;
    p.d = D.d;
    p.scale = D.scale;
    int exponent = 0;
    p.scale_m = 2.f * std::frexp(D.scale, &exponent);
    p.scale_pow = std::ldexp(1.f, exponent - 1);
    p.scale2 = (float)((double)D.scale * fs::kLog2ed);
    p.planes = L.planes;
    p.plane_x = p.plane_w = L.dp;
    p.x = L.pack_x ? base + L.px : x;
    p.ldx = L.pack_x ? (long long)L.planes * L.dp : D.ldx;
    p.ldw = L.pack_w ? (long long)L.planes * L.dp : D.ldw;
    p.lddx = D.lddx;
    p.lddw = D.lddw;
    p.ignore = D.ignore_index;
    p.part = reinterpret_cast<float2 *>(base + L.part);
    p.hit = reinterpret_cast<float *>(base + L.hit);
    p.dl = base + L.dl;
    p.ld_dl = L.ld_dl;
    p.acc = reinterpret_cast<float *>(base + L.acc);
    p.ld_acc = L.ld_acc;
    p.parts = L.parts;
    p.timeout_ns = kTimeoutNs;
    p.err = dev.err;
    return p;
}

// The piece of the classes from c0 on: its rows of w, copied into planes where the products need that.
fs_status xent_piece(const fs_xent_desc &D, const XentPlan &L, const void *w, void *ws, int c0, fs::XentParams &p,
                     cudaStream_t s) {
    const bool bf16 = D.dtype == FS_BF16;
    const char *rows = static_cast<const char *>(w) + D.ldw * c0 * (bf16 ? 2 : 4);
    p.c0 = c0;
    p.c1 = std::min(D.v, c0 + L.piece);
    p.w = rows;
    if (L.pack_w) {
        p.w = static_cast<char *>(ws) + L.pw;
        OPS_LAUNCH(fs::launch_xent_pack(rows, D.ldw, p.c1 - c0, D.d, L.dp, bf16, static_cast<char *>(ws) + L.pw, s), 1);
    }
    return FS_OK;
}

}  // namespace

extern "C" {

size_t fs_cross_attn_workspace(const fs_attn_desc *desc, int grad) {
    Device dev;
    if (check_attn(desc, grad != 0) != FS_OK) return 0;
    if (current_device(&dev) != FS_OK) return SIZE_MAX;
    return attn_workspace(*desc, grad != 0, dev);
}

fs_status fs_cross_attn(const fs_attn_desc *desc, const void *q, const void *k, const void *v, const int *k_len,
                        const float *bias, void *out, float *lse, void *workspace, size_t workspace_bytes,
                        void *stream) {
    fs_status st = check_attn(desc, false);
    if (st != FS_OK) return st;
    const fs_attn_desc &D = *desc;
    if (D.batch == 0 || D.n == 0) return FS_OK;
    if (!q || !out || (D.m > 0 && (!k || !v))) return reject(FS_ERR_INVALID_ARG, "null argument");
    Device dev;
    if ((st = current_device(&dev)) != FS_OK) return st;
    const bool bf16 = D.dtype == FS_BF16, tc = attn_tc(D, q, k, v, out);
    const int rows = D.n * (D.heads / D.kv_heads);
    const bool few = !tc && fs::xattn_token_ok(q, D.q, k, D.k, v, D.v, D.d, D.dv, rows, bf16);
    const AttnKind kind = tc ? kTensor : few ? kToken : kSimt;
    const AttnPlan L = plan_attn(D, false, kind, k_len != nullptr, dev);
    if ((st = check_workspace(workspace, workspace_bytes, L.total)) != FS_OK) return st;
    fs::AttnParams p = attn_params(D, L, dev, workspace);
    p.q = q;
    p.k = k;
    p.v = v;
    p.k_len = k_len;
    p.bias = bias;
    p.out = out;
    p.lse = lse;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tc)
        OPS_LAUNCH(fs::launch_xattn_tc(p, s), 1);
    else
        OPS_LAUNCH(fs::launch_xattn_simt(p, bf16, s), 1);
    if (p.splits > 1) OPS_LAUNCH(fs::launch_xattn_combine(p, bf16, s), 1);
    return FS_OK;
}

fs_status fs_cross_attn_grad(const fs_attn_desc *desc, const void *q, const void *k, const void *v, const int *k_len,
                             const float *bias, const void *out, const float *lse, const void *dout, void *dq,
                             void *dk, void *dv, void *workspace, size_t workspace_bytes, void *stream) {
    fs_status st = check_attn(desc, true);
    if (st != FS_OK) return st;
    const fs_attn_desc &D = *desc;
    if (D.batch == 0 || (D.n == 0 && D.m == 0)) return FS_OK;
    if ((D.n > 0 && (!q || !out || !lse || !dout || !dq)) || (D.m > 0 && (!k || !v || !dk || !dv)))
        return reject(FS_ERR_INVALID_ARG, "null argument");
    Device dev;
    if ((st = current_device(&dev)) != FS_OK) return st;
    const bool tc = attn_grad_tc(D, q, k, v, dout, dq, dk, dv);
    const AttnPlan L = plan_attn(D, true, tc ? kTensor : kSimt, false, dev);
    if ((st = check_workspace(workspace, workspace_bytes, L.total)) != FS_OK) return st;
    fs::AttnParams p = attn_params(D, L, dev, workspace);
    p.q = q;
    p.k = k;
    p.v = v;
    p.k_len = k_len;
    p.bias = bias;
    p.out = const_cast<void *>(out);
    p.lse = const_cast<float *>(lse);
    p.dout = dout;
    p.dq = dq;
    p.dk = dk;
    p.dv_out = dv;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = D.dtype == FS_BF16;
    if (!bias || D.n == 0) p.top = nullptr;
    if (p.top) {
        const AttnPlan F = plan_attn(D, false, tc ? kTensor : kSimt, false, dev);
        fs::AttnParams f = p;
        f.stats = 1;
        f.unit_rows = F.unit_rows;
        f.blocks = F.blocks;
        f.main_units = F.blocks * D.kv_heads * D.batch;  // none is split
        f.splits = 1;
        OPS_LAUNCH(tc ? fs::launch_xattn_tc(f, s) : fs::launch_xattn_simt(f, bf16, s), 1);
    }
    if (D.n > 0) OPS_LAUNCH(fs::launch_xattn_dot(p, bf16, s), 1);
    if (tc) {
        OPS_LAUNCH(fs::launch_xattn_grad_tc(p, s), 1);
        if (L.key_parts > 1 || L.row_parts > 1) OPS_LAUNCH(fs::launch_xattn_grad_join(p, s), 1);
    } else {
        OPS_LAUNCH(fs::launch_xattn_grad_simt(p, bf16, dev.sms, s), 1);
        if (L.key_parts > 1 || L.row_parts > 1) OPS_LAUNCH(fs::launch_xattn_grad_join_simt(p, bf16, s), 1);
    }
    return FS_OK;
}

size_t fs_cross_entropy_workspace(const fs_xent_desc *desc, const void *x, const void *w, int grad) {
    Device dev;
    if (check_xent(desc, grad != 0) != FS_OK) return 0;
    if (current_device(&dev) != FS_OK) return SIZE_MAX;
    return plan_xent(*desc, x, w, grad != 0, dev).total;
}

fs_status fs_cross_entropy(const fs_xent_desc *desc, const void *x, const void *w, const long long *target,
                           float *loss, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    fs_status st = check_xent(desc, false);
    if (st != FS_OK) return st;
    const fs_xent_desc &D = *desc;
    if (D.n == 0) return FS_OK;
    if (!x || !w || !target || !loss || !lse) return reject(FS_ERR_INVALID_ARG, "null argument");
    Device dev;
    if ((st = current_device(&dev)) != FS_OK) return st;
    const XentPlan L = plan_xent(D, x, w, false, dev);
    if ((st = check_workspace(workspace, workspace_bytes, L.total)) != FS_OK) return st;
    fs::XentParams p = xent_params(D, L, dev, workspace, x);
    p.target = target;
    p.loss = loss;
    p.lse = lse;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (L.pack_x)
        OPS_LAUNCH(fs::launch_xent_pack(x, D.ldx, D.n, D.d, L.dp, D.dtype == FS_BF16, const_cast<void *>(p.x), s), 1);
    for (int c0 = 0; c0 < D.v; c0 += L.piece) {
        if ((st = xent_piece(D, L, w, workspace, c0, p, s)) != FS_OK) return st;
        OPS_LAUNCH(fs::launch_xent_lse(p, dev.pairs, s), 1);
    }
    OPS_LAUNCH(fs::launch_xent_finish(p, L.tiles, s), 1);
    return FS_OK;
}

fs_status fs_cross_entropy_grad(const fs_xent_desc *desc, const void *x, const void *w, const long long *target,
                                const float *lse, const float *dloss, const float *dlse, void *dx, void *dw,
                                void *workspace, size_t workspace_bytes, void *stream) {
    fs_status st = check_xent(desc, true);
    if (st != FS_OK) return st;
    const fs_xent_desc &D = *desc;
    if (!w || !dw || (D.n > 0 && (!x || !target || !lse || !dloss || !dx)))
        return reject(FS_ERR_INVALID_ARG, "null argument");
    Device dev;
    if ((st = current_device(&dev)) != FS_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = D.dtype == FS_BF16;
    const size_t elem = bf16 ? 2 : 4;
    if (D.n == 0) {
        cudaError_t e = cudaMemset2DAsync(dw, (D.v > 1 ? (size_t)D.lddw : (size_t)D.d) * elem, 0, D.d * elem, D.v, s);
        return e == cudaSuccess ? FS_OK : reject(FS_ERR_CUDA, "cudaMemset2DAsync: %s", cudaGetErrorString(e));
    }
    const XentPlan L = plan_xent(D, x, w, true, dev);
    if ((st = check_workspace(workspace, workspace_bytes, L.total)) != FS_OK) return st;
    fs::XentParams p = xent_params(D, L, dev, workspace, x);
    p.target = target;
    p.lse = const_cast<float *>(lse);
    p.dloss = dloss;
    p.dlse = dlse;
    p.dx = dx;
    if (L.pack_x)
        OPS_LAUNCH(fs::launch_xent_pack(x, D.ldx, D.n, D.d, L.dp, bf16, const_cast<void *>(p.x), s), 1);
    for (int c0 = 0; c0 < D.v; c0 += L.piece) {
        if ((st = xent_piece(D, L, w, workspace, c0, p, s)) != FS_OK) return st;
        p.acc_add = c0 > 0;
        p.dw = static_cast<char *>(dw) + D.lddw * c0 * (long long)elem;
        OPS_LAUNCH(fs::launch_xent_dl(p, dev.pairs, s), 1);
        OPS_LAUNCH(fs::launch_xent_dx(p, L.direct, dev.pairs, s), 1);
        const int rows = bf16 ? D.n : fs::kXentF32Terms;
        for (int r0 = 0; r0 < D.n; r0 += rows)
            OPS_LAUNCH(fs::launch_xent_dw(p, r0, std::min(D.n, r0 + rows), r0 > 0, dev.pairs, s), 1);
    }
    if (!L.direct) OPS_LAUNCH(fs::launch_xent_reduce(p, bf16, s), 1);
    return FS_OK;
}

fs_status fs_selftest_check(int timeout_ms, void *stream) {
    if (timeout_ms < 1) return reject(FS_ERR_INVALID_ARG, "timeout_ms must be >= 1");
    Device dev;
    fs_status st = current_device(&dev);
    if (st != FS_OK) return st;
    OPS_LAUNCH(fs::launch_wait_probe((unsigned long long)timeout_ms * 1000000ull, dev.err,
                                     static_cast<cudaStream_t>(stream)), 1);
    return FS_OK;
}

fs_status fs_check(void *stream) {
    Device dev;
    fs_status st = current_device(&dev);
    if (st != FS_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    static std::mutex mu;  // one check at a time has the word of taken bits
    int bits = 0;
    cudaError_t e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) {
        std::lock_guard<std::mutex> lock(mu);
        take_errors_kernel<<<1, 1, 0, s>>>();
        e = cudaGetLastError();
        if (e == cudaSuccess) fs::count_launches(1);
        if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(&bits, g_ops_taken, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    if (e != cudaSuccess) return reject(FS_ERR_CUDA, "fs_check: %s", cudaGetErrorString(e));
    if (bits & fs::kDevErrTimeout) return reject(FS_ERR_TIMEOUT, "a bounded device wait timed out");
    return FS_OK;
}

}  // extern "C"
