/*
 * Stands in for the library's calls that the module sv_torch makes (preloaded
 * before it): each is counted, launches nothing and returns stand_in_status.
 * Calls that are made through the library's own handle are not met.
 */
int PyGILState_Check(void);

int stand_in_status, stand_in_calls, stand_in_with_gil;

static int taken(void) {
  ++stand_in_calls;
  stand_in_with_gil += PyGILState_Check();
  return stand_in_status;
}

int sv_rms_norm(void) { return taken(); }
int sv_rms_norm_fp8(void) { return taken(); }
int sv_rms_norm_backward(void) { return taken(); }
int sv_grad_norm(void) { return taken(); }
int sv_clip_grad_norm(void) { return taken(); }
