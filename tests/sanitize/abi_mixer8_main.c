/* Malformed calls of the delta rule, the RMS norm and the 8-bit rows: each
 * returns an error (or BIMAMBA_OK for an empty problem) without any HIP call. */
#include <stdio.h>
#include <string.h>

#include "bimamba.h"

static int bad = 0;
#define EXPECT(code, call)                                                    \
    do {                                                                      \
        int rc_ = (call);                                                     \
        if (rc_ != (code)) { printf("line %d: %d\n", __LINE__, rc_); bad = 1; } \
    } while (0)

int main(void) {
    void *p = (void *)(uintptr_t)0x10000, *odd = (void *)(uintptr_t)0x10002;
    float *f = (float *)p;
    size_t n = 0;
    static int32_t cu[1001];
    bimamba_rows8 r = {p, f}, none = {0, 0};
    bimamba_shape s;
    bimamba_delta_dir d, empty;
    bimamba_delta_grad g, gone;
    memset(&s, 0, sizeof s);
    memset(&empty, 0, sizeof empty);
    memset(&gone, 0, sizeof gone);
    s.batch = 1; s.seqlen = 100; s.nheads = 2; s.headdim = 16; s.d_state = 16; s.ngroups = 1; s.chunk = 64;
    s.dtype = BIMAMBA_BF16;
    d.q = d.k = d.v = p; d.g = d.beta = f;
    g.dq = g.dk = g.dv = g.dg = g.dbeta = f;
    for (int i = 0; i <= 1000; ++i) cu[i] = i / 10;

    EXPECT(BIMAMBA_EINVAL, bimamba_delta_workspace_size(0, 0, 0, &n));
    EXPECT(BIMAMBA_EINVAL, bimamba_delta_workspace_size(&s, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_delta_workspace_size(&s, 0, -1, &n));
    EXPECT(BIMAMBA_OK, bimamba_delta_workspace_size(&s, 1, 1000, &n));
    EXPECT(BIMAMBA_OK, bimamba_delta_bwd_workspace_size(&s, 1000, &n));
    EXPECT(BIMAMBA_EINVAL, bimamba_delta_fwd(&s, 0, 0, 1.f, 0, 0, 0, 0, f, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_delta_fwd(&s, &empty, 0, 1.f, 0, 0, 0, 0, f, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_delta_fwd(&s, &d, &empty, 1.f, 0, 0, 0, 0, f, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_delta_fwd(&s, &d, 0, 1.f, 0, 0, 0, 0, 0, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_delta_fwd(&s, &d, 0, 1.f / 0.f, 0, 0, 0, 0, f, 0, 0, 0));
    EXPECT(BIMAMBA_EWORKSPACE, bimamba_delta_fwd(&s, &d, &d, 1.f, 0, 0, 0, 0, f, 0, 0, 0));
    EXPECT(BIMAMBA_EWORKSPACE, bimamba_delta_fwd(&s, &d, 0, 1.f, cu, 1000, 0, 0, f, p, 16, 0));
    cu[500] = 99;
    EXPECT(BIMAMBA_EINVAL, bimamba_delta_fwd(&s, &d, 0, 1.f, cu, 1000, 0, 0, f, p, 1 << 30, 0));
    cu[500] = 50;
    EXPECT(BIMAMBA_EINVAL, bimamba_delta_step(&s, 0, &d, 0, 1.f, 1, f, p, 1 << 30, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_delta_bwd(&s, &d, 0, 1.f, 0, 0, 0, 0, f, 0, 0, 0, p, 1 << 30, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_delta_bwd(&s, &d, 0, 1.f, 0, 0, 0, 0, f, &gone, 0, 0, p, 1 << 30, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_delta_bwd(&s, &d, 0, 1.f, 0, 0, 0, 0, f, &g, &g, 0, p, 1 << 30, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_delta_bwd(&s, &d, 0, 1.f, 0, 0, 0, 0, 0, &g, 0, 0, p, 1 << 30, 0));
    EXPECT(BIMAMBA_EWORKSPACE, bimamba_delta_bwd(&s, &d, &d, 1.f, 0, 0, 0, 0, f, &g, &g, 0, 0, 0, 0));
    s.seqlen = 0;
    EXPECT(BIMAMBA_OK, bimamba_delta_fwd(&s, &empty, 0, 1.f, 0, 0, 0, 0, 0, 0, 0, 0));
    s.seqlen = 2147483647;
    s.batch = 2147483647;
    EXPECT(BIMAMBA_EUNSUPPORTED, bimamba_delta_workspace_size(&s, 1, 0, &n));
    EXPECT(BIMAMBA_EUNSUPPORTED, bimamba_delta_bwd_workspace_size(&s, 2147483647, &n));

    EXPECT(BIMAMBA_EINVAL, bimamba_rms_norm(4, 64, BIMAMBA_BF16, p, 0, f, 0.f, 0, 0, f, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_rms_norm(4, 64, BIMAMBA_BF16, p, p, f, 0.f, p, 0, f, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_rms_norm(4, 64, BIMAMBA_BF16, p, 0, f, 0.f, 0, 0, f, &none, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_rms_norm(4, 64, BIMAMBA_F32, odd, 0, f, 0.f, p, 0, f, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_rms_norm(4, 64, BIMAMBA_F32, p, 0, f, -1.f, p, 0, f, 0, 0));
    EXPECT(BIMAMBA_OK, bimamba_rms_norm(0, 64, BIMAMBA_BF16, 0, 0, 0, 0.f, 0, 0, 0, 0, 0));
    EXPECT(BIMAMBA_OK, bimamba_rms_norm_bwd_workspace_size(2147483647LL, 16384, BIMAMBA_F32, &n));
    EXPECT(BIMAMBA_EINVAL, bimamba_rms_norm_bwd(4, 64, BIMAMBA_BF16, 0, 0, f, f, p, 0, p, 0, 0, 0, 0));
    EXPECT(BIMAMBA_EWORKSPACE, bimamba_rms_norm_bwd(4, 64, BIMAMBA_BF16, p, 0, f, f, p, 0, p, f, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_rows8_pack(4, 64, BIMAMBA_BF16, p, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_rows8_pack(4, 64, BIMAMBA_BF16, p, &none, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_linear8(4, 64, 8, BIMAMBA_BF16, 0, &r, 0, p, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_linear8(4, 64, 8, BIMAMBA_BF16, &r, &none, 0, p, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_linear8(4, 64, 8, BIMAMBA_BF16, &r, &r, 0, p, 0));
    EXPECT(BIMAMBA_EUNSUPPORTED, bimamba_linear8(2147483647LL, 64, 1 << 24, BIMAMBA_BF16, &r, &r, 0, p, 0));
    EXPECT(BIMAMBA_OK, bimamba_linear8(0, 64, 8, BIMAMBA_BF16, &r, &r, 0, 0, 0));
    if (!bad) printf("abi mixer checks: ok\n");
    return bad;
}
