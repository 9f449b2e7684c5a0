/* Malformed calls of the training entry points: each returns an error (or
 * BIMAMBA_OK for an empty problem) without any HIP call. */
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
    uint8_t *u = (uint8_t *)p;
    size_t n = 0;
    int32_t cu[131];
    bimamba_act8 a = {p, p}, none = {0, 0};
    bimamba_conv_shape s;
    bimamba_conv_dir d;
    bimamba_conv_grad g;
    memset(&s, 0, sizeof s);
    memset(&d, 0, sizeof d);
    memset(&g, 0, sizeof g);
    memset(cu, 0, sizeof cu);
    cu[130] = 8;
    s.batch = 1; s.seqlen = 8; s.nheads = 2; s.headdim = 16; s.d_state = 16; s.ngroups = 1; s.width = 4;
    s.dtype = BIMAMBA_BF16; s.activation = 1;
    d.weight = f; d.x = p; d.B = p; d.C = p;
    g.xbc = p; g.weight = f; g.dx = f; g.dB = f; g.dC = f; g.dxbc = p; g.dweight = f;

    EXPECT(BIMAMBA_EINVAL, bimamba_act8_pack(-1, 32, BIMAMBA_BF16, p, &a, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_act8_pack(1, 32, BIMAMBA_BF16, p, &none, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_act8_unpack(1, 32, BIMAMBA_F32, &a, odd, 0));
    EXPECT(BIMAMBA_EUNSUPPORTED, bimamba_act8_unpack(1, 0, BIMAMBA_F32, &a, p, 0));
    EXPECT(BIMAMBA_OK, bimamba_act8_unpack(0, 1, BIMAMBA_F32, 0, 0, 0));

    EXPECT(BIMAMBA_EINVAL, bimamba_conv1d_act8(0, &d, &a, 0, 0, 0, 0, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_conv1d_act8(&s, 0, &a, 0, 0, 0, 0, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_conv1d_act8(&s, &d, &none, 0, 0, 0, 0, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_conv1d_act8(&s, &d, &a, &d, 0, 0, 0, 0, 0, 0));
    EXPECT(BIMAMBA_EWORKSPACE, bimamba_conv1d_act8(&s, &d, &a, 0, 0, cu, 130, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_conv1d_act8_workspace_size(&s, 1, 0));
    EXPECT(BIMAMBA_OK, bimamba_conv1d_act8_workspace_size(&s, 130, &n));

    EXPECT(BIMAMBA_EINVAL, bimamba_conv1d_bwd(0, &g, 0, 0, 0, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_conv1d_bwd(&s, 0, 0, 0, 0, 0, 0, 0));
    EXPECT(BIMAMBA_EWORKSPACE, bimamba_conv1d_bwd(&s, &g, 0, 0, 0, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_conv1d_bwd(&s, &g, &g, 0, 0, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_conv1d_bwd(&s, &g, 0, 0, 1, 0, 0, 0));
    EXPECT(BIMAMBA_EWORKSPACE, bimamba_conv1d_bwd(&s, &g, 0, cu, 130, p, 16, 0));
    EXPECT(BIMAMBA_OK, bimamba_conv1d_bwd_workspace_size(&s, 1, 130, &n));
    s.seqlen = (1 << 30) + 1;
    EXPECT(BIMAMBA_EUNSUPPORTED, bimamba_conv1d_bwd_workspace_size(&s, 1, 0, &n));
    s.seqlen = 1 << 20;
    s.batch = 2000;
    EXPECT(BIMAMBA_EUNSUPPORTED, bimamba_conv1d_bwd_workspace_size(&s, 1, 0, &n));

    EXPECT(BIMAMBA_EUNSUPPORTED, bimamba_gated_norm_bwd_workspace_size(1, 100, 100, BIMAMBA_F32, &n));
    EXPECT(BIMAMBA_OK, bimamba_gated_norm_bwd_workspace_size(2147483647LL, 8192, 8192, BIMAMBA_F32, &n));
    EXPECT(BIMAMBA_EWORKSPACE,
           bimamba_gated_norm_bwd(4, 512, 256, BIMAMBA_BF16, p, u, p, u, f, 0.f, p, f, p, f, 0, 0, 0));
    EXPECT(BIMAMBA_EINVAL,
           bimamba_gated_norm_bwd(4, 512, 256, BIMAMBA_BF16, odd, u, p, u, f, 0.f, p, f, p, f, 0, 0, 0));

    EXPECT(BIMAMBA_EINVAL, bimamba_layer_norm(4, 64, BIMAMBA_BF16, p, p, f, f, 0.f, p, 0, f, f, 0, 0));
    EXPECT(BIMAMBA_EINVAL, bimamba_layer_norm(4, 64, BIMAMBA_BF16, p, 0, f, f, 0.f, p, 0, f, f, &none, 0));
    EXPECT(BIMAMBA_EUNSUPPORTED, bimamba_layer_norm(4, 16385, BIMAMBA_BF16, p, 0, f, f, 0.f, p, 0, f, f, &a, 0));
    EXPECT(BIMAMBA_OK, bimamba_layer_norm_bwd_workspace_size(2147483647LL, 16384, BIMAMBA_F32, &n));
    EXPECT(BIMAMBA_EWORKSPACE,
           bimamba_layer_norm_bwd(4, 64, BIMAMBA_F32, p, u, f, f, f, p, p, p, f, f, p, 1, 0));
    if (!bimamba_last_error()[0]) bad = 1;
    printf(bad ? "abi training checks: FAILED\n" : "abi training checks: ok\n");
    return bad;
}
