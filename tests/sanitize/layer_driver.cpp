// Drives the host side of kda_layer_abi.cpp under AddressSanitizer / UndefinedBehaviorSanitizer:
// every status, the workspace sizes, and the plan of segments (how the chunks of any batch are
// divided, and that the workspace holds what the plan says).  Prints "layer driver ok".
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>

#include "../../gated_delta_rule_log2_amd/csrc/kda_layer.h"
#include "../../include/kda.h"

extern int g_stub_launches;
extern kda::SsmParams g_ssm;

static int failures = 0;
#define EXPECT(cond, what)                                       \
    do {                                                         \
        if (!(cond)) {                                           \
            std::printf("FAIL %s (line %d)\n", what, __LINE__); \
            ++failures;                                          \
        }                                                        \
    } while (0)

static kda_ssm_desc ssm(int32_t B, int32_t T, int32_t H, int32_t G, int32_t N, int32_t P) {
    kda_ssm_desc d;
    std::memset(&d, 0, sizeof(d));
    d.B = B; d.T = T; d.H = H; d.G = G; d.N = N; d.P = P; d.num_seqs = B;
    d.x_dtype = d.dt_dtype = KDA_DTYPE_BF16;
    d.x_stride = (int64_t)H * P; d.dt_stride = H; d.b_stride = d.c_stride = (int64_t)G * N;
    return d;
}

static uint32_t seed = 1;
static uint32_t rnd(uint32_t n) { return (seed = seed * 1664525u + 1013904223u) / 65536u % n; }

// A call of fwd or bwd with every pointer inside buffers of their own (nothing reads them).
static kda_status call(const kda_ssm_desc &d, bool bwd, const int64_t *cu, void *ws, size_t bytes) {
    static char one[64], two[64];
    void *F = one;
    float *f = reinterpret_cast<float *>(one), *g = reinterpret_cast<float *>(two);
    if (!bwd) return kda_ssm_fwd(&d, F, F, f, F, F, f, f, f, cu, F, g, ws, bytes, nullptr);
    return kda_ssm_bwd(&d, F, F, f, F, F, f, f, f, cu, F, f, F, F, f, F, F, f, f, g, ws, bytes, nullptr);
}

// Chunks and segments of the plan against the batch, counted here.
static void plan(kda_ssm_desc d, const std::vector<int64_t> &cu, bool bwd) {
    if (!cu.empty()) d.num_seqs = (int32_t)cu.size() - 1, d.cu_seqlens_host = cu.data();
    size_t bytes = 0;
    const kda_status st = bwd ? kda_ssm_bwd_workspace_size(&d, &bytes) : kda_ssm_fwd_workspace_size(&d, &bytes);
    EXPECT(st == KDA_OK && bytes > 0, "workspace");
    if (st != KDA_OK || bytes > (1u << 30)) return;
    std::vector<char> ws(bytes);
    const int64_t *dev = cu.empty() ? nullptr : cu.data();
    EXPECT(call(d, bwd, dev, ws.data(), bytes - 1) == KDA_ERR_WORKSPACE, "one byte less");
    EXPECT(call(d, bwd, dev, ws.data(), bytes) == KDA_OK, "call");
    const int L = d.x_dtype == KDA_DTYPE_BF16 ? 64 : 32;
    int64_t chunks = 0, segs = 0, most = 1;
    EXPECT(g_ssm.seg >= 1, "segment length");
    for (int32_t n = 0; n < d.num_seqs; ++n) {
        const int64_t len = cu.empty() ? d.T : cu[n + 1] - cu[n], c = (len + L - 1) / L;
        const int64_t s = c > g_ssm.seg ? (c + g_ssm.seg - 1) / g_ssm.seg : 1;
        chunks += c;
        segs += s;
        if (s > most) most = s;
    }
    EXPECT(g_ssm.total_chunks == chunks && g_ssm.total_segs == segs && g_ssm.max_segs == most, "counts");
    EXPECT((g_ssm.seg_state != nullptr) == (most > 1), "states of segments where there are several");
    // the last region of either layout ends inside the workspace
    auto inside = [&](const float *p, size_t n) {
        const char *b = reinterpret_cast<const char *>(p), *e = b + n * sizeof(float);
        return b >= ws.data() && e <= ws.data() + bytes;
    };
    const size_t state = (size_t)d.N * d.P, ch = (size_t)chunks * d.H;
    EXPECT(inside(g_ssm.d, ch * L) && inside(g_ssm.ch, ch * L) && inside(g_ssm.cl, ch * L), "decays");
    if (most > 1) EXPECT(inside(g_ssm.seg_state, (bwd ? 2 : 1) * segs * d.H * state) && inside(g_ssm.seg_dec, (bwd ? 2 : 1) * segs * d.H), "segments");
    if (bwd) {
        EXPECT(inside(g_ssm.last_state, d.num_seqs * d.H * state) && inside(g_ssm.w_o, ch * L * (d.N / 16)) &&
                   inside(g_ssm.w_q, ch * L * (d.N / 16)) && inside(g_ssm.w_dot, segs * d.H * (d.N / 16)) &&
                   inside(g_ssm.sums, ch * 4) && inside(g_ssm.w_decay, ch), "terms");
        const int hg = d.H / d.G;
        EXPECT(g_ssm.split >= 1 && g_ssm.split <= hg && (hg + g_ssm.split - 1) / g_ssm.split <= 2, "at most two heads to a part");
        EXPECT((hg + g_ssm.split - 1) / g_ssm.split * (g_ssm.split - 1) < hg, "no part without a head");
        if (g_ssm.split > 1) EXPECT(inside(g_ssm.dCp, (size_t)g_ssm.split * d.B * d.T * d.G * d.N), "parts");
    }
}

int main() {
    for (int bwd = 0; bwd < 2; ++bwd) {
        for (int32_t T : {0, 1, 63, 64, 65, 128, 129, 1000, 8192, 100000})
            for (int32_t H : {1, 2, 3, 8, 30, 511, 512, 700}) {
                if ((int64_t)T * H > 1000000) continue;
                plan(ssm(1, T, H, H % 3 ? 1 : 3, 32, 64), {}, bwd);
                plan(ssm(7, T / 7, H, H, 32, 32), {}, bwd);
                kda_ssm_desc f = ssm(2, T / 2, H, 1, 64, 32);
                f.x_dtype = KDA_DTYPE_FP32;
                plan(f, {}, bwd);
            }
        for (int k = 0; k < 400; ++k) {
            const int32_t T = 1 + rnd(6000), n = 1 + rnd(k < 40 ? 600 : 40), H = 1 + rnd(k % 3 ? 8 : 70);
            std::vector<int64_t> cu(n + 1);
            for (int32_t i = 1; i < n; ++i) cu[i] = rnd(T + 1);
            cu[n] = T;
            for (int32_t i = 1; i < n; ++i)
                for (int32_t j = i; j > 1 && cu[j] < cu[j - 1]; --j) { const int64_t t = cu[j]; cu[j] = cu[j - 1]; cu[j - 1] = t; }
            plan(ssm(1, T, H, 1, 32, 32), cu, bwd);
        }
        plan(ssm(1 << 16, 1, 4, 1, 32, 32), {}, bwd);
    }

    kda_ssm_desc d = ssm(1, 256, 4, 2, 64, 64);
    size_t bytes = 0;
    struct Case { const char *what; void (*edit)(kda_ssm_desc &); kda_status want; };
    const int64_t bad[3] = {0, 300, 256}, good[2] = {0, 256};
    static const int64_t *offsets;
    const Case cases[] = {
        {"B 0", [](kda_ssm_desc &x) { x.B = 0; }, KDA_ERR_SHAPE},
        {"T < 0", [](kda_ssm_desc &x) { x.T = -1; }, KDA_ERR_SHAPE},
        {"tokens past 2^30", [](kda_ssm_desc &x) { x.B = 1 << 16; x.T = 1 << 16; x.num_seqs = x.B; }, KDA_ERR_SHAPE},
        {"N 48", [](kda_ssm_desc &x) { x.N = 48; }, KDA_ERR_UNSUPPORTED},
        {"P 160", [](kda_ssm_desc &x) { x.P = 160; }, KDA_ERR_UNSUPPORTED},
        {"flags", [](kda_ssm_desc &x) { x.flags = 2; }, KDA_ERR_UNSUPPORTED},
        {"groups", [](kda_ssm_desc &x) { x.G = 3; }, KDA_ERR_GVA},
        {"x stride", [](kda_ssm_desc &x) { x.x_stride = 255; }, KDA_ERR_SHAPE},
        {"dt stride", [](kda_ssm_desc &x) { x.dt_stride = 3; }, KDA_ERR_SHAPE},
        {"x stride past 2^24", [](kda_ssm_desc &x) { x.x_stride = 1 << 24; }, KDA_ERR_SHAPE},
        {"C stride past 2^24", [](kda_ssm_desc &x) { x.c_stride = 1 << 24; }, KDA_ERR_SHAPE},
        {"heads past 2^24", [](kda_ssm_desc &x) { x.H = x.G = 1 << 18; x.x_stride = 1 << 24; x.dt_stride = 1 << 18; }, KDA_ERR_SHAPE},
        {"sequences", [](kda_ssm_desc &x) { x.num_seqs = 2; }, KDA_ERR_SHAPE},
        {"offsets", [](kda_ssm_desc &x) { x.num_seqs = 2; x.cu_seqlens_host = offsets; }, KDA_ERR_VARLEN},
        {"dtype", [](kda_ssm_desc &x) { x.dt_dtype = 7; }, KDA_ERR_DTYPE},
    };
    offsets = bad;
    for (const Case &c : cases) {
        kda_ssm_desc e = d;
        c.edit(e);
        EXPECT(kda_ssm_fwd_workspace_size(&e, &bytes) == c.want, c.what);
        EXPECT(kda_ssm_bwd_workspace_size(&e, &bytes) == c.want, c.what);
    }
    EXPECT(kda_ssm_fwd_workspace_size(nullptr, &bytes) == KDA_ERR_NULL_POINTER, "null descriptor");
    EXPECT(kda_ssm_bwd_workspace_size(&d, nullptr) == KDA_ERR_NULL_POINTER, "null size");
    EXPECT(kda_ssm_bwd_workspace_size(&d, &bytes) == KDA_OK, "size");
    std::vector<char> ws(bytes);
    EXPECT(call(d, true, good, ws.data(), bytes) == KDA_ERR_VARLEN, "device offsets alone");
    EXPECT(call(d, false, nullptr, nullptr, bytes) == KDA_ERR_WORKSPACE, "no workspace");
    EXPECT(call(d, true, nullptr, ws.data(), bytes) == KDA_OK, "backward");

    kda_conv_desc c;
    std::memset(&c, 0, sizeof(c));
    c.B = 2; c.T = 100; c.D = 24; c.W = 4; c.num_seqs = 2; c.x_stride = 24;
    EXPECT(kda_short_conv_bwd_workspace_size(&c, &bytes) == KDA_OK && bytes == 4u * 4 * 5 * 24, "convolution's size");
    c.x_stride = 23;
    EXPECT(kda_short_conv_bwd_workspace_size(&c, &bytes) == KDA_ERR_SHAPE, "convolution's stride");
    kda_norm_desc n;
    std::memset(&n, 0, sizeof(n));
    n.rows = 5; n.D = 40; n.eps = 1e-6f;
    EXPECT(kda_rms_norm_bwd_workspace_size(&n, &bytes) == KDA_OK && bytes == 4u * 5 * 40, "norm's size");
    n.D = kda::kNormMaxD + 1;
    EXPECT(kda_rms_norm_bwd_workspace_size(&n, &bytes) == KDA_ERR_UNSUPPORTED, "norm's width");
    EXPECT(g_stub_launches > 0, "launches");

    if (failures) return 1;
    std::printf("layer driver ok\n");
    return 0;
}
